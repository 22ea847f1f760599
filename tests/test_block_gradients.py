"""MoeBlock's forward and backward with a bias for the choice, and without a residual: against the oracle
and against central differences in 64 bits at the same choice."""
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
T, H, I, E, K = 60, 256, 128, 16, 3


def _t(rng, *s, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).bfloat16().to(DEV)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                               ("sigmoid", False)])
@pytest.mark.parametrize("residual", [False, True])
def test_block_with_a_bias(score, renormalize, residual):
    rng = np.random.default_rng(8)
    bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32)).to(DEV)
    bias[5] = -float("inf")  # an expert that nobody gets
    b = MoeBlock(1 + _t(rng, H, scale=0.1), _t(rng, E, H, scale=0.1), _t(rng, E, 2 * I, H, scale=H ** -0.5),
                 _t(rng, E, H, I, scale=I ** -0.5), K, bias=bias, score=score, renormalize=renormalize, scale=1.5)
    x, res = _t(rng, T, H), _t(rng, T, H) if residual else None
    out, h, saved = b.forward(x, res)
    y, logits, ids = saved[1], saved[3], saved[4]
    z32, b32 = logits.float().cpu().numpy(), bias.cpu().numpy()
    rid, rw = ob.moe_route(z32, b32, K, score, renormalize, 1.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    assert not (rid == 5).any() and (rid != ob.moe_route(z32, None, K, score, renormalize, 1.5)[0]).any()
    W1, W2, gate, gamma = (util.f64(t) for t in (b.W1, b.W2, b.gate, b.gamma))
    # A, each expert's output and the logits are rounded to bf16 on the way
    util.assert_close(out, ob.moe_decode(util.f64(y), rid, rw, W1, W2)[0], "forward", rel=2e-2, abs_rms=2e-2)
    x64, r64 = util.f64(x), util.f64(res) if residual else 0.0
    util.assert_close(h, x64 + r64, "residual stream")
    got_d, h2 = b.decode(x, res)
    assert torch.equal(h, h2)
    util.assert_close(got_d, util.f64(out), "decode against forward")
    dout, dh = _t(rng, T, H), _t(rng, T, H)
    d64, dh64 = util.f64(dout), util.f64(dh)
    g = b.backward(dout, dh, saved)
    mask = np.where(np.isneginf(b32), -np.inf, 0.0)

    def loss(x64, gamma, gate, W1, W2):
        s, y, _ = ob.add_rmsnorm(x64, r64, gamma, b.eps)
        z = y @ gate.T
        total = np.sum(s * dh64)
        for t in range(T):
            a = ob._row_scores(z[t], z[t] + mask, score)
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
    assert not g["dW1"][5].any() and not g["dgate"][5].any()
