"""MoeBlock with its further parts -- experts with biases and a shifted SwiGLU, a shared expert, the joint
with the block before (norm, gate, dropout, scales) -- in training against the fp64 oracle and central
differences, and in decoding against its own training path."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from oracle import linear as ol
import util

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
from precision_grouped_gemm_gb300.block import MoeBlock  # noqa: E402

DEV = "cuda"
H, I, S, E, K = 256, 128, 192, 16, 3


def _t(rng, *s, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).bfloat16().to(DEV)


def _block(seed, biased=True, shared=True, join=True, fmt=None, dropout=0.2):
    rng = np.random.default_rng(seed)
    kw = {}
    if biased:
        kw.update(b1=_t(rng, E, 2 * I), b2=_t(rng, E, H), alpha=1.702, offset=1.0, swiglu_limit=2.5)
    if shared:
        kw.update(S1=_t(rng, 2 * S, H, scale=H ** -0.5), S2=_t(rng, H, S, scale=S ** -0.5))
    if join:
        kw.update(gamma_post=1 + _t(rng, H, scale=0.1), residual_scale=0.9, branch_scale=0.7, dropout=dropout)
    return rng, MoeBlock(1 + _t(rng, H, scale=0.1), _t(rng, E, H, scale=0.1), _t(rng, E, 2 * I, H, scale=H ** -0.5),
                         _t(rng, E, H, I, scale=I ** -0.5), K, fmt=fmt, **kw)


def _output(b, v, y, ids, w, form):
    """The block's output from its norm's in 64 bits, at a choice."""
    out = np.zeros((y.shape[0], H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t):
            a = ol.linear(y[t], v["W1"][e:e + 1], [len(t)], v["b1"][e:e + 1], None, "swiglu", **form)[0]
            out[t] += w[t, j][:, None] * (a @ v["W2"][e].T + v["b2"][e])
    a = ol.linear(y, v["S1"][None], [y.shape[0]], None, None, "swiglu", **form)[0]
    return out + a @ v["S2"].T


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["row", "column"])
def test_block_with_all_parts(gate):
    rng, b = _block(3)
    T = 60
    x, res = _t(rng, T, H), _t(rng, T, H)
    g_in = torch.rand(T, device=DEV) + 0.5 if gate == "row" else 1 + _t(rng, H, scale=0.3)
    state = torch.tensor([123, -9], device=DEV)
    out, h, saved = b.forward(x, res, gate=g_in, rng=state)
    form = {"alpha": 1.702, "offset": 1.0, "limit": 2.5}
    names = ("x", "residual", "gamma_post", "gamma", "gate", "W1", "W2", "b1", "b2", "S1", "S2", "gate_in")
    v = {n: util.f64(t) if t.dtype == torch.bfloat16 else t.double().cpu().numpy()
         for n, t in zip(names, (x, res, b.gamma_post, b.gamma, b.gate, b.W1, b.W2, b.b1, b.b2, b.S1, b.S2, g_in))}
    mask = ol.keep(T, H, 0.2, (123, -9))

    def run(v, rid=None):
        gin = v["gate_in"][:, None] if gate == "row" else v["gate_in"]
        s, y, _, _ = ol.join(v["x"], v["residual"], v["gamma_post"], v["gamma"], gin, 0.9, 0.7, 0.2, mask, b.eps)
        z = y @ v["gate"].T
        if rid is None:
            rid = saved[4].cpu().numpy()
        a = np.exp(z - z.max(axis=1, keepdims=True))
        w = np.take_along_axis(a, rid, 1)
        return s, _output(b, v, y, rid, w / w.sum(axis=1, keepdims=True), form)

    rid, _ = ob.moe_route(saved[3].float().cpu().numpy(), None, K, "softmax", True, 1.0)
    np.testing.assert_array_equal(saved[4].cpu().numpy(), rid)
    s, ref = run(v)
    util.assert_close(h, s, "residual stream")
    # y, the logits, A, each expert's output and their sum are rounded to bf16 on the way
    util.assert_close(out, ref, "forward", rel=2e-2, abs_rms=2e-2)
    dout, dh = _t(rng, T, H), _t(rng, T, H)
    g = b.backward(dout, dh, saved)
    d64, dh64 = util.f64(dout), util.f64(dh)

    def loss(v):
        s, o = run(v)
        return np.sum(s * dh64) + np.sum(o * d64)

    for name in names:
        got = g["d" + name].double().cpu().numpy()
        assert got.shape == v[name].shape, name
        d = np.where(got > 0, 1.0, -1.0) * np.abs(rng.standard_normal(got.shape))  # every term adds up
        up, dn = dict(v), dict(v)
        up[name], dn[name] = v[name] + 1e-5 * d, v[name] - 1e-5 * d
        assert np.sum(got * d) == pytest.approx((loss(up) - loss(dn)) / 2e-5, rel=2e-2), name


@pytest.mark.gpu
@pytest.mark.parametrize("biased,shared,join", [(True, False, False), (True, True, True), (False, True, False),
                                                (False, False, True), (False, True, True)])
@pytest.mark.parametrize("T", [1, 9, 100])
def test_block_decode_equals_forward(T, biased, shared, join):
    rng, b = _block(5, biased, shared, join, dropout=0.0)
    x, res = _t(rng, T, H), _t(rng, T, H)
    gate = torch.rand(T, device=DEV) if join else None
    out, h, _ = b.forward(x, res, gate=gate)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, h2 = b.decode(x, res, err=err, gate=gate)
    assert pgg.read_error(err) == 0 and torch.equal(h, h2)
    # the training path rounds the activation, each expert's output and their sum to bf16
    util.assert_close(got, util.f64(out), "decode against forward", rel=2e-2, abs_rms=2e-2)
    again, _ = b.decode(x, res, gate=gate)
    assert torch.equal(got, again)
    b.check_decode()


@pytest.mark.gpu
def test_block_decode_with_parts_in_a_graph():
    for biased in (False, True):
        rng, b = _block(6, biased)
        x, res, gate = _t(rng, 5, H), _t(rng, 5, H), torch.rand(5, device=DEV)
        b.prepare_decode()
        ref, _ = b.decode(x, res, gate=gate)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got, _ = b.decode(x, res, gate=gate)
        for _ in range(2):
            got.zero_()
            graph.replay()
            assert torch.equal(got, ref)
            x.copy_(_t(rng, 5, H))
            ref, _ = b.decode(x, res, gate=gate)
        b.check_decode()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,tol", [("e4m3", 0.08), ("e2m1", 0.4)])
def test_block_mx_decode_with_parts(fmt, tol):
    # (the tolerances of the MX decode without these parts, which add only bf16 products)
    rng, b = _block(7, biased=False, fmt=fmt, dropout=0.0)
    x, res, gate = _t(rng, 33, H), _t(rng, 33, H), torch.rand(33, device=DEV)
    got, h = b.decode(x, res, gate=gate)
    ref, h2, _ = b.forward(x, res, gate=gate)
    assert torch.equal(h, h2)
    assert 0 < float((got.double() - ref.double()).norm() / ref.double().norm()) < tol


def test_block_refusals():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    args = (z(H), z(E, H), z(E, 2 * I, H), z(E, H, I), K)
    with pytest.raises(ValueError, match="MX"):
        MoeBlock(*args, fmt="e4m3", b1=z(E, 2 * I))
    with pytest.raises(ValueError, match="MX"):
        MoeBlock(*args, fmt="e2m1", alpha=1.5)
    with pytest.raises(ValueError, match="S1"):
        MoeBlock(*args, S1=z(2 * S, H))
    with pytest.raises(ValueError, match="rng"):
        MoeBlock(*args, dropout=0.1).forward(z(2, H))
