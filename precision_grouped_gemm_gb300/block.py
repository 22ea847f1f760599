"""A MoE block around the expert layer: norm, gate, routing, experts, in its two uses.

Training (`MoeBlock.forward` / `backward`) goes the long way, over the permuted batch and the grouped
GEMMs; decoding (`MoeBlock.decode`, up to 128 tokens) hands the norm's output straight to the
few-token layer: three small kernels and one weight stream.  With `fmt` the decode weights are MX
operands, quantized when the block is made and again when W1 or W2 have changed, and the norm emits
the MX operand of its tokens itself.

    s = x + residual, y = rmsnorm(s) gamma     add_rmsnorm
    logits = y gate^T, in fp32                 grouped_linear
    ids, w = top-k of the logits               moe_route
    out = sum_j w_j expert_{ids_j}(y)          moe_permute ... moe_combine, or moe_decode

A block may have more parts, each left out unless it is given:

    biases b1, b2 of the experts, and a SwiGLU g sigmoid(alpha g) (u + offset)     grouped_linear
    a shared expert S1, S2 that every token takes, added to out                    grouped_linear
    s = residual_scale residual + branch_scale gate dropout(rmsnorm(x) gamma_post) block_join

with their gradients (grouped_linear_bwd, block_join_bwd).  The few-token layer has no biases: a block
with them decodes the long way, on bf16 weights.
"""
from __future__ import annotations

import dataclasses
import weakref

import torch

from . import _binding as B


def _gone():
    return None


def _version(t):
    return None if t.is_inference() else t._version


@dataclasses.dataclass
class MoeBlock:
    gamma: torch.Tensor        # [H] bf16
    gate: torch.Tensor         # [E, H] bf16, E % 8 == 0
    W1: torch.Tensor           # [E, 2I, H] bf16 (gate | up)
    W2: torch.Tensor           # [E, H, I] bf16
    k: int
    bias: torch.Tensor = None  # [E] fp32: added to the logits for the choice only
    score: str = "softmax"
    renormalize: bool = True
    scale: float = 1.0
    swiglu_limit: float = 0.0
    eps: float = 1e-6
    fmt: str = None            # decode weights: None (bf16), "e4m3" or "e2m1"
    b1: torch.Tensor = None    # [E, 2I] bf16: the experts' biases
    b2: torch.Tensor = None    # [E, H] bf16
    alpha: float = 1.0         # of the SwiGLU, as in grouped_linear
    offset: float = 0.0
    S1: torch.Tensor = None    # [2S, H] bf16 (gate | up): a shared expert, with the same SwiGLU
    S2: torch.Tensor = None    # [H, S] bf16
    gamma_post: torch.Tensor = None  # [H] bf16: the norm of x before it joins the residual stream
    residual_scale: float = 1.0
    branch_scale: float = 1.0
    dropout: float = 0.0       # of x, in training

    def __post_init__(self):
        E, I2, H = self.W1.shape
        self.sizes = E, H, I2 // 2
        # (a form that the few-token layer and the fused expert products do not have)
        self._biased = self.b1 is not None or self.b2 is not None or self.alpha != 1.0 or self.offset != 0.0
        if self._biased and self.fmt is not None:
            raise ValueError("MX decode weights go with neither biases nor alpha and offset")
        if (self.S1 is None) != (self.S2 is None):
            raise ValueError("a shared expert needs S1 and S2")
        self._mx = self._mx_of = self._ws = None
        self._err = torch.zeros(1, dtype=torch.int32, device=self.W1.device)
        self.quantize_weights()

    def _one_group(self, rows, device):
        return torch.full((1,), rows, dtype=torch.int32, device=device)

    def _route(self, y, err=None):
        # (fp32: rounded to bf16, logits tie, and move an expert's weight by 2^-8 of the logit)
        logits, _ = B.grouped_linear(y, self.gate, out_dtype=torch.float32, err=err)
        ids, w = B.moe_route(logits, self.k, self.bias, self.score, self.renormalize, self.scale)
        return logits, ids, w

    def _form(self):
        return {"act": "swiglu", "alpha": self.alpha, "offset": self.offset, "limit": self.swiglu_limit}

    def _joined(self, gate):
        return (gate is not None or self.gamma_post is not None or self.residual_scale != 1.0 or self.branch_scale != 1.0
                or self.dropout)

    def _join(self, gate, rng=None):
        """block_join's arguments besides the tensors that flow; rng None: no dropout."""
        return {"gamma_post": self.gamma_post, "gamma": self.gamma, "gate": gate, "residual_scale": self.residual_scale,
                "branch_scale": self.branch_scale, "p": 0.0 if rng is None else self.dropout, "rng": rng}

    def _experts(self, Xs, lens, save, err=None):
        """The experts' outputs for the permuted batch -> (Ys, A, Hs)."""
        if self._biased:
            A, Hs = B.grouped_linear(Xs, self.W1, lens, bias=self.b1, save_z=save, err=err, **self._form())
            return B.grouped_linear(A, self.W2, lens, bias=self.b2, err=err)[0], A, Hs
        A, Hs = B.grouped_fc1_swiglu(Xs, self.W1, lens, swiglu_limit=self.swiglu_limit, save_h=save, err=err)
        return B.grouped_gemm_fwd(A, self.W2, lens, err=err), A, Hs

    def _shared(self, y, out, save, err=None):
        """Adds the shared expert's output to `out`, in place -> (As, Zs)."""
        if self.S1 is None:
            return None, None
        As, Zs = B.grouped_linear(y, self.S1, save_z=save, err=err, **self._form())
        B.grouped_linear(As, self.S2, residual=out, Y=out, err=err)
        return As, Zs

    def forward(self, x, residual=None, gate=None, rng=None):
        """-> (out [T,H], h [T,H]: the new residual stream, saved tensors for `backward`).

        gate: fp32 [T] or bf16 [H], of x; rng: int64 [2] on the device, (seed, offset) of the dropout, of which
        `saved` has a copy: the caller may step it on before `backward`."""
        E, _, _ = self.sizes
        if self.dropout and rng is None:
            raise ValueError("dropout needs rng")
        rng = rng.clone() if self.dropout else None
        joined = self._joined(gate)
        if joined:
            h, y, _, _, rstd_post, rstd = B.block_join(x, residual, eps=self.eps, **self._join(gate, rng))
        else:
            rstd_post = None
            h, y, _, _, rstd = B.add_rmsnorm(x, residual, self.gamma, self.eps)
        logits, ids, w = self._route(y)
        Xs, lens, pos = B.moe_permute(ids, y, E)
        Ys, A, Hs = self._experts(Xs, lens, True)
        out = B.moe_combine(Ys, pos, w)
        As, Zs = self._shared(y, out, True)
        # (a block that only adds x keeps it no longer than the caller does)
        return out, h, (h, y, rstd, logits, ids, w, Xs, lens, pos, A, Hs, Ys, x if joined else None, rstd_post, gate, rng,
                        As, Zs)

    def backward(self, dout, dh, saved):
        """Gradients of `forward` -> dict: dx, dresidual (dx itself in a block that only adds the two), dgamma,
        dgate, dW1, dW2, and of the parts that the block has: db1, db2, dS1, dS2, dgamma_post, and dgate_in of
        forward's gate."""
        h, y, rstd, logits, ids, w, Xs, lens, pos, A, Hs, Ys, x, rstd_post, gate, rng, As, Zs = saved
        one = self._one_group(y.shape[0], y.device)
        g = {}
        dYs, dw = B.moe_combine_bwd(dout, Ys, pos, w)
        if self._biased:
            dH, db1 = B.grouped_linear_bwd(B.grouped_gemm_dgrad(dYs, self.W2, lens), Hs, lens, **self._form())
            if self.b1 is not None:
                g["db1"] = db1
            if self.b2 is not None:
                g["db2"] = B.grouped_linear_bwd(dYs, group_lens=lens)[1]
        else:
            dH = B.grouped_fc2_dgrad_swiglu_bwd(dYs, self.W2, Hs, lens, swiglu_limit=self.swiglu_limit)
        g["dW2"] = B.grouped_gemm_wgrad(A, dYs, lens)
        g["dW1"] = B.grouped_gemm_wgrad(Xs, dH, lens)
        dy = B.moe_combine(B.grouped_gemm_dgrad(dH, self.W1, lens), pos)
        if self.S1 is not None:
            dZs, _ = B.grouped_linear_bwd(B.grouped_gemm_dgrad(dout, self.S2[None], one), Zs, **self._form())
            g["dS2"] = B.grouped_gemm_wgrad(As, dout, one)[0]
            g["dS1"] = B.grouped_gemm_wgrad(y, dZs, one)[0]
            dy += B.grouped_gemm_dgrad(dZs, self.S1[None], one)
        dlogits = B.moe_route_bwd(logits, ids, dw, self.bias, self.score, self.renormalize, self.scale).bfloat16()
        g["dgate"] = B.grouped_gemm_wgrad(y, dlogits, one)[0]
        dy += B.grouped_gemm_dgrad(dlogits, self.gate[None], one)
        if self._joined(gate):
            g["dx"], g["dresidual"], dgp, g["dgamma"], dgi = B.block_join_bwd(dy, dh, x, h, rstd_post, rstd,
                                                                              **self._join(gate, rng))
            if dgp is not None:
                g["dgamma_post"] = dgp
            if dgi is not None:
                g["dgate_in"] = dgi
        else:
            g["dx"], g["dgamma"] = B.add_rmsnorm_bwd(dy, dh, h, self.gamma, rstd)
            g["dresidual"] = g["dx"]
        return g

    def decode(self, x, residual=None, err=None, gate=None):
        """`forward` for up to 128 tokens, inference only (no dropout) -> (out, h).  A block has one workspace, so its
        decode calls run in the order of one stream.  err: the caller's error word; without one the block's
        own, which `check_decode` reads.  A first call inside a graph's capture has a workspace of the
        graph's, zeroed at every replay: call `prepare_decode` before the capture to avoid that."""
        err = self._err if err is None else err
        if self._biased:
            h, y, _, _ = self._entry(x, residual, gate)
            _, ids, w = self._route(y, err)
            Xs, lens, pos = B.moe_permute(ids, y, self.sizes[0], err=err)
            out = B.moe_combine(self._experts(Xs, lens, False, err)[0], pos, w)
            self._shared(y, out, False, err)
            return out, h
        ws = self._ws
        if ws is None:
            # (memory of a graph's pool is the graph's: eager calls and other graphs get their own)
            ws = self._workspace() if torch.cuda.is_current_stream_capturing() else self.prepare_decode()
        if self.fmt is not None:
            mx = self._mx
            if not self._current():
                # (a capture quantizes into its own memory, at every replay)
                mx = self._quantized() if torch.cuda.is_current_stream_capturing() else self.quantize_weights()
        h, y, codes, scales = self._entry(x, residual, gate)
        _, ids, w = self._route(y, err)
        if self.fmt is None:
            out = B.moe_decode(y, ids, w, self.W1, self.W2, swiglu_limit=self.swiglu_limit, ws=ws, err=err)
        else:
            out = B.mx_moe_decode(self.fmt, codes, scales, ids, w, *mx, swiglu_limit=self.swiglu_limit, ws=ws, err=err)
        self._shared(y, out, False, err)
        return out, h

    def _entry(self, x, residual, gate):
        """What stands in front of a decoding block's gate -> (h, y, codes, scales)."""
        if self._joined(gate):
            return B.block_join(x, residual, eps=self.eps, fmt=self.fmt, save_rstd=False, **self._join(gate))[:4]
        return B.add_rmsnorm(x, residual, self.gamma, self.eps, fmt=self.fmt, save_rstd=False)[:4]

    def _quantized(self, into=(None,) * 4):
        E, H, I = self.sizes
        return (*B.mx_quantize_rowwise_blocked(self.W1.view(E * 2 * I, H), self.fmt, *into[:2]),
                *B.mx_quantize_rowwise_blocked(self.W2.view(E * H, I), self.fmt, *into[2:]))

    def _current(self):
        """Whether the MX operands are those of W1 and W2: the same tensors, not written to since.  (A decoding
        block may give up its bf16 weights: with W1 or W2 None the operands are what there is.)"""
        if self.W1 is None or self.W2 is None:
            return True
        return all(ref() is t and version == _version(t) for (ref, version), t in zip(self._mx_of, (self.W1, self.W2)))

    def __getstate__(self):  # references to tensors by identity do not travel: a copy quantizes anew
        return {**self.__dict__, "_mx_of": [(_gone, None)] * 2}

    def quantize_weights(self):
        """The MX operands of W1 and W2 as they are now (fmt), in the memory of the ones before: decode calls
        this itself after a change that torch counts.  For changes that it does not (`.data`, kernels that write
        through an address, inference tensors), and before replays of a captured decode, the caller does.
        Without fmt decode reads W1 and W2 themselves, and this does nothing."""
        if self.fmt is None:
            return None
        self._mx = self._quantized(self._mx or (None,) * 4)
        self._mx_of = [(weakref.ref(t), _version(t)) for t in (self.W1, self.W2)]
        return self._mx

    def _workspace(self):
        E, H, I = self.sizes
        return B.moe_decode_workspace(128, self.k, H, I, E, self.fmt, self.gamma.device)

    def prepare_decode(self):
        """Makes the decode workspace, which is kept for the block's life: every call leaves it ready for
        the next.  A workspace that is there is zeroed, which it needs after a timeout."""
        if self._ws is None:
            self._ws = self._workspace()
        else:
            self._ws.zero_()
        return self._ws

    def check_decode(self):
        """Raises PggError if a decode call without an error word of the caller's has failed since the last
        check, with the block ready again.  Waits for the current stream."""
        code = B.read_error(self._err)
        if code:
            self._err.zero_()
            if self._ws is not None:
                self.prepare_decode()
            raise B.PggError(code, "MoeBlock.decode")
