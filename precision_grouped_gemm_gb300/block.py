"""A MoE block around the expert layer: norm, gate, routing, experts, in its two uses.

Training (`MoeBlock.forward` / `backward`) goes the long way, over the permuted batch and the grouped
GEMMs; decoding (`MoeBlock.decode`, up to 128 tokens) hands the norm's output straight to the
few-token layer: three small kernels and one weight stream.  With `fmt` the decode weights are MX
operands, quantized when the block is made and again when W1 or W2 have changed, and the norm emits
the MX operand of its tokens itself.

    s = x + residual, y = rmsnorm(s) gamma     add_rmsnorm
    logits = y gate^T                          grouped_gemm_fwd with one group
    ids, w = top-k of the logits               moe_route
    out = sum_j w_j expert_{ids_j}(y)          moe_permute ... moe_combine, or moe_decode
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

    def __post_init__(self):
        E, I2, H = self.W1.shape
        self.sizes = E, H, I2 // 2
        self._mx = self._mx_of = self._ws = None
        self._err = torch.zeros(1, dtype=torch.int32, device=self.W1.device)
        self.quantize_weights()

    def _one_group(self, rows, device):
        return torch.full((1,), rows, dtype=torch.int32, device=device)

    def _route(self, y):
        logits = B.grouped_gemm_fwd(y, self.gate[None], self._one_group(y.shape[0], y.device))
        ids, w = B.moe_route(logits, self.k, self.bias, self.score, self.renormalize, self.scale)
        return logits, ids, w

    def forward(self, x, residual=None):
        """-> (out [T,H], h [T,H]: the new residual stream, saved tensors for `backward`)."""
        E, _, _ = self.sizes
        h, y, _, _, rstd = B.add_rmsnorm(x, residual, self.gamma, self.eps)
        logits, ids, w = self._route(y)
        Xs, lens, pos = B.moe_permute(ids, y, E)
        A, Hs = B.grouped_fc1_swiglu(Xs, self.W1, lens, swiglu_limit=self.swiglu_limit)
        Ys = B.grouped_gemm_fwd(A, self.W2, lens)
        return B.moe_combine(Ys, pos, w), h, (h, y, rstd, logits, ids, w, Xs, lens, pos, A, Hs, Ys)

    def backward(self, dout, dh, saved):
        """Gradients of `forward` -> dict: dx (of x and of residual), dgamma, dgate, dW1, dW2."""
        h, y, rstd, logits, ids, w, Xs, lens, pos, A, Hs, Ys = saved
        one = self._one_group(y.shape[0], y.device)
        dYs, dw = B.moe_combine_bwd(dout, Ys, pos, w)
        dH = B.grouped_fc2_dgrad_swiglu_bwd(dYs, self.W2, Hs, lens, swiglu_limit=self.swiglu_limit)
        dW2 = B.grouped_gemm_wgrad(A, dYs, lens)
        dW1 = B.grouped_gemm_wgrad(Xs, dH, lens)
        dy = B.moe_combine(B.grouped_gemm_dgrad(dH, self.W1, lens), pos)
        dlogits = B.moe_route_bwd(logits, ids, dw, self.bias, self.score, self.renormalize, self.scale)
        dgate = B.grouped_gemm_wgrad(y, dlogits, one)[0]
        dy += B.grouped_gemm_dgrad(dlogits, self.gate[None], one)
        dx, dgamma = B.add_rmsnorm_bwd(dy, dh, h, self.gamma, rstd)
        return {"dx": dx, "dgamma": dgamma, "dgate": dgate, "dW1": dW1, "dW2": dW2}

    def decode(self, x, residual=None, err=None):
        """`forward` for up to 128 tokens, inference only -> (out, h).  A block has one workspace, so its
        decode calls run in the order of one stream.  err: the caller's error word; without one the block's
        own, which `check_decode` reads.  A first call inside a graph's capture has a workspace of the
        graph's, zeroed at every replay: call `prepare_decode` before the capture to avoid that."""
        err = self._err if err is None else err
        ws = self._ws
        if ws is None:
            # (memory of a graph's pool is the graph's: eager calls and other graphs get their own)
            ws = self._workspace() if torch.cuda.is_current_stream_capturing() else self.prepare_decode()
        if self.fmt is not None:
            mx = self._mx
            if not self._current():
                # (a capture quantizes into its own memory, at every replay)
                mx = self._quantized() if torch.cuda.is_current_stream_capturing() else self.quantize_weights()
        h, y, codes, scales, _ = B.add_rmsnorm(x, residual, self.gamma, self.eps, fmt=self.fmt, save_rstd=False)
        _, ids, w = self._route(y)
        if self.fmt is None:
            return B.moe_decode(y, ids, w, self.W1, self.W2, swiglu_limit=self.swiglu_limit, ws=ws, err=err), h
        return B.mx_moe_decode(self.fmt, codes, scales, ids, w, *mx, swiglu_limit=self.swiglu_limit, ws=ws,
                               err=err), h

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
