"""The MoE block (norm, gate, routing, experts) in training and in decoding, on the GPU."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from oracle import grouped_gemm as og
import util

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
from precision_grouped_gemm_gb300.block import MoeBlock  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _block(T, H, I, E, k, seed, fmt=None, **kw):
    rng = np.random.default_rng(seed)
    t = lambda *s, scale=1.0: torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).bfloat16().to(DEV)  # noqa: E731
    b = MoeBlock(1 + t(H, scale=0.1), t(E, H, scale=0.1), t(E, 2 * I, H, scale=H ** -0.5), t(E, H, I, scale=I ** -0.5), k,
                 fmt=fmt, **kw)
    return b, t(T, H), t(T, H), rng


def _oracle_out(b, y, logits, limit=None, fmt=None):
    """The block's output from its own bf16 norm output and logits, in fp64."""
    ids, w = ob.moe_route(logits.float().cpu().numpy(), None if b.bias is None else b.bias.cpu().numpy(), b.k, b.score,
                          b.renormalize, b.scale)
    return ids, w, ob.moe_decode(util.f64(y), ids, w, util.f64(b.W1), util.f64(b.W2), limit, fmt)[0]


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_block_forward_and_backward(score, renormalize):
    b, x, res, rng = _block(60, 256, 128, 16, 3, 1, score=score, renormalize=renormalize, scale=1.5)
    out, h, saved = b.forward(x, res)
    y, logits, ids = saved[1], saved[3], saved[4]
    rid, _, ref = _oracle_out(b, y, logits)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    # A, each expert's output and the logits are rounded to bf16 on the way
    util.assert_close(out, ref, "block forward", rel=2e-2, abs_rms=2e-2)
    s, ry, _ = ob.add_rmsnorm(util.f64(x), util.f64(res), util.f64(b.gamma), b.eps)
    util.assert_close(h, s, "residual stream")
    util.assert_close(y, ry, "norm")
    dout, dh = (torch.from_numpy(rng.standard_normal((60, 256)).astype(np.float32)).bfloat16().to(DEV) for _ in range(2))
    g = b.backward(dout, dh, saved)
    # central differences of the whole block in fp64 at the same choice, along one direction of each input
    W1, W2, gate, gamma = (util.f64(t) for t in (b.W1, b.W2, b.gate, b.gamma))
    x64, r64, d64, dh64 = util.f64(x), util.f64(res), util.f64(dout), util.f64(dh)

    def loss(x64, gamma, gate, W1, W2):
        s, y, _ = ob.add_rmsnorm(x64, r64, gamma, b.eps)
        z = y @ gate.T
        total = np.sum(s * dh64)
        for t in range(60):
            a = ob._row_scores(z[t], z[t], score)
            Z = a[rid[t]].sum() if renormalize else a.sum() if score == "softmax" else 1.0
            o = sum(1.5 * a[e] / Z * (W2[e] @ og.swiglu_fwd((W1[e] @ y[t])[None])[0]) for e in rid[t])
            total += np.sum(o * d64[t])
        return total

    for i, name in enumerate(["dx", "dgamma", "dgate", "dW1", "dW2"]):
        args = [x64, gamma, gate, W1, W2]
        got = g[name].double().cpu().numpy()
        v = np.where(got > 0, 1.0, -1.0) * np.abs(rng.standard_normal(got.shape))  # every term adds up
        e = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + e * v, args[i] - e * v
        num = (loss(*up) - loss(*dn)) / (2 * e)
        assert np.sum(got * v) == pytest.approx(num, rel=2e-2), name


@pytest.mark.parametrize("T", [1, 7, 64])
def test_block_decode_equals_forward(T):
    b, x, res, _ = _block(T, 512, 256, 32, 4, 2, swiglu_limit=1.0)
    out, h, _ = b.forward(x, res)
    got, h2 = b.decode(x, res)
    assert torch.equal(h, h2)
    util.assert_close(got, util.f64(out), "decode against forward")
    again, _ = b.decode(x, res)
    assert torch.equal(got, again)


@pytest.mark.parametrize("fmt,tol", [("e4m3", 0.08), ("e2m1", 0.4)])
def test_block_mx_decode_is_near_bf16(fmt, tol):
    # two quantized products: an e4m3 element is off by up to 2^-4 of itself (2.3% rms with the scale's
    # headroom), an e2m1 one by up to 1/4 (about 12% rms), on each of four operands
    b, x, res, _ = _block(33, 512, 256, 16, 2, 3, fmt=fmt)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, _ = b.decode(x, res, err=err)
    assert pgg.read_error(err) == 0
    ref, _, _ = b.forward(x, res)
    d = (got.double() - ref.double()).norm() / ref.double().norm()
    assert 0 < float(d) < tol
