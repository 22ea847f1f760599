"""CPU checks of the operators around the grouped GEMMs: the oracle against differences and closed
forms, and the entry points' refusals (no GPU, no compute call)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import block as ob


def _rng(*seed):
    return np.random.default_rng(list(seed))


def _difference(f, x, d, step=1e-5):
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


def test_rmsnorm_closed_forms():
    s, y, rstd = ob.add_rmsnorm(np.array([[3.0, -4.0]]), None, np.array([1.0, 2.0]), 0.0)
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), -8 / np.sqrt(12.5)]], rtol=1e-15)
    _, y2, _ = ob.add_rmsnorm(np.array([[1.0, -1.0]]), np.array([[2.0, -3.0]]), np.array([1.0, 2.0]), 0.0)
    np.testing.assert_array_equal(y, y2)
    _, y0, r0 = ob.add_rmsnorm(np.zeros((1, 4)), None, np.ones(4), 0.25)  # a zero row
    assert not y0.any() and r0[0] == 2.0


def test_rmsnorm_gradients_against_differences():
    r = _rng(1)
    R, C, eps = 5, 24, 1e-3
    x, gamma, dy, dh = r.normal(size=(R, C)), r.normal(size=C), r.normal(size=(R, C)), r.normal(size=(R, C))

    def loss(x, gamma):
        s, y, _ = ob.add_rmsnorm(x, None, gamma, eps)
        return np.sum(y * dy) + np.sum(s * dh)

    _, _, rstd = ob.add_rmsnorm(x, None, gamma, eps)
    dx, dgamma = ob.add_rmsnorm_bwd(dy, dh, x, gamma, rstd)
    for i in range(4):
        v, g = r.normal(size=(R, C)), r.normal(size=C)
        assert np.sum(dx * v) == pytest.approx(_difference(lambda z: loss(z, gamma), x, v), rel=1e-7)
        assert np.sum(dgamma * g) == pytest.approx(_difference(lambda z: loss(x, z), gamma, g), rel=1e-7)


def test_route_closed_forms():
    x = np.array([[1.0, 3.0, 3.0, -np.inf]], dtype=np.float32)
    ids, w = ob.moe_route(x, None, 2, "softmax", True, 2.0)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[1.0, 1.0]])          # a tie: the lowest first
    ids, w = ob.moe_route(x, None, 4, "softmax", False, 1.0)
    assert ids.tolist() == [[1, 2, 0, 3]] and w[0, 3] == 0.0 and np.isclose(w.sum(), 1.0)
    ids, w = ob.moe_route(x, np.array([9.0, 0, 0, 0]), 1, "sigmoid", False, 1.0)
    assert ids.tolist() == [[0]] and np.isclose(w[0, 0], 1 / (1 + np.exp(-1.0)))  # the bias only chooses
    ids, w = ob.moe_route(np.full((1, 5), -np.inf, np.float32), None, 3, "softmax", False, 1.0)
    assert ids.tolist() == [[0, 1, 2]] and not w.any()                        # a row that is masked whole
    ids, w = ob.moe_route(np.array([[0.0, np.nan, 1.0]], np.float32), None, 2, "softmax", True, 1.0)
    assert ids.tolist() == [[2, 0]] and np.isnan(w).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(score, renormalize):
    r = _rng(2)
    T, E, k = 6, 12, 3
    x = r.normal(size=(T, E))
    x[1, 3] = -np.inf
    ids, _ = ob.moe_route(x, None, k, score, renormalize, 2.5)
    dw, v = r.normal(size=(T, k)), r.normal(size=(T, E))
    v[1, 3] = 0.0

    def loss(z):  # in fp64, at a fixed choice
        total = 0.0
        for t in range(T):
            a = ob._row_scores(z[t], z[t], score)
            Z = a[ids[t]].sum() if renormalize else a.sum() if score == "softmax" else 1.0
            total += np.sum(2.5 * dw[t] * a[ids[t]] / Z)
        return total

    x = x.astype(np.float32).astype(np.float64)  # what the oracle's keys are made of
    d = ob.moe_route_bwd(x, None, ids, dw, score, renormalize, 2.5)
    assert np.sum(d * v) == pytest.approx(_difference(loss, x, v), rel=1e-7)
    assert d[1, 3] == 0.0


def test_decode_is_a_sum_over_choices():
    r = _rng(3)
    T, k, E, H, I = 3, 2, 4, 8, 32
    x, W1, W2 = r.normal(size=(T, H)), r.normal(size=(E, 2 * I, H)), r.normal(size=(E, H, I))
    ids = np.array([[0, 3], [2, 2], [1, 7]])  # a repeated expert, and one that does not exist
    w = r.random(size=(T, k))
    out, _, _ = ob.moe_decode(x, ids, w, W1, W2, limit=1.0)
    for t in range(T):
        ref = np.zeros(H)
        for j in range(k):
            if ids[t, j] >= E:
                continue
            hid = [sum(W1[ids[t, j], i, c] * x[t, c] for c in range(H)) for i in range(2 * I)]
            g, u = np.minimum(hid[:I], 1.0), np.clip(hid[I:], -1.0, 1.0)
            ref += w[t, j] * (W2[ids[t, j]] @ (g / (1 + np.exp(-g)) * u))
        np.testing.assert_allclose(out[t], ref, rtol=1e-12)
    q, _, _ = ob.moe_decode(x, ids[:1], w[:1], W1, W2, fmt="e4m3")
    assert 0 < np.linalg.norm(q[0] - ob.moe_decode(x, ids[:1], w[:1], W1, W2)[0][0]) / np.linalg.norm(q[0]) < 0.1


# ---------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    from precision_grouped_gemm_gb300 import _binding, build
    build.build()
    return _binding.lib()


G = 1 << 20  # an aligned address that is never followed
P = ctypes.c_void_p


def test_norm_refusals(lib):
    def fwd(x=G, r=G, g=G, R=4, C=64, eps=1e-6, fmt=1, h=G, y=G, codes=G, scales=G, rstd=G):
        return lib.pgg_add_rmsnorm(x, r, g, R, C, eps, fmt, h, y, codes, scales, rstd, None)
    assert fwd(R=0) == 0                          # no rows: nothing to do
    assert fwd(x=None) == 1 and fwd(g=None) == 1
    assert fwd(R=-1) == 1 and fwd(C=16384 + 32) == 1 and fwd(C=0) == 1
    assert fwd(C=72) == 3                         # codes need whole blocks of 32
    assert fwd(C=68, fmt=0, codes=None, scales=None) == 3
    assert fwd(fmt=7) == 1 and fwd(fmt=0) == 1    # unknown format; codes without a format
    assert fwd(scales=None) == 1
    assert fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1
    assert fwd(fmt=0, codes=None, scales=None, h=None, y=None, rstd=None) == 1  # no output
    assert fwd(x=G + 8) == 3 and fwd(rstd=G + 2) == 3
    size = ctypes.c_size_t(0)
    assert lib.pgg_add_rmsnorm_bwd_workspace_size(10, 64, ctypes.byref(size)) == 0 and size.value >= 10 * 64 * 4
    assert lib.pgg_add_rmsnorm_bwd_workspace_size(10, 60, ctypes.byref(size)) == 3

    def bwd(dy=G, dh=G, h=G, g=G, rstd=G, R=10, C=64, dx=G, dg=G, ws=G, n=1 << 20):
        return lib.pgg_add_rmsnorm_bwd(dy, dh, h, g, rstd, R, C, dx, dg, ws, n, None)
    assert bwd(n=64) == 1 and bwd(ws=None) == 1   # workspace too small, absent
    assert bwd(dg=None) == 1 and bwd(h=None) == 1 and bwd(dx=G + 4) == 3 and bwd(C=12) == 3


def test_route_refusals(lib):
    def fwd(x=G, dt=0, b=None, T=5, E=16, k=2, sc=0, rn=1, scale=1.0, ids=G, w=G):
        return lib.pgg_moe_route(x, dt, b, T, E, k, sc, rn, scale, ids, w, None)
    assert fwd(T=0) == 0
    assert fwd(dt=2) == 1 and fwd(sc=2) == 1 and fwd(rn=2) == 1
    assert fwd(E=0) == 1 and fwd(E=1025) == 1 and fwd(k=0) == 1 and fwd(k=17) == 1 and fwd(E=64, k=33) == 1
    assert fwd(scale=float("nan")) == 1 and fwd(scale=float("inf")) == 1
    assert fwd(x=None) == 1 and fwd(ids=None) == 1 and fwd(w=None) == 1
    assert fwd(x=G + 4) == 3 and fwd(b=G + 1) == 3 and fwd(w=G + 2) == 3 and fwd(T=1 << 26) == 1
    assert lib.pgg_moe_route_bwd(G, 0, None, G, None, 5, 16, 2, 0, 1, 1.0, G, None) == 1
    assert lib.pgg_moe_route_bwd(G, 0, None, G, G, 5, 16, 2, 0, 1, 1.0, G + 4, None) == 3
    assert lib.pgg_moe_route_bwd(G, 0, None, G, G, 0, 16, 2, 0, 1, 1.0, None, None) == 0


def test_decode_refusals(lib):
    size = ctypes.c_size_t(0)
    assert lib.pgg_moe_decode_workspace_size(0, 4, 2, 256, 128, 8, ctypes.byref(size)) == 0
    need = size.value

    def run(x=G, ids=G, w=G, w1=G, w2=G, out=G, T=4, k=2, H=256, I=128, E=8, lim=0.0, ws=G, n=need, err=None):
        return lib.pgg_moe_decode(x, ids, w, w1, w2, out, T, k, H, I, E, lim, ws, n, err, None)
    assert run(T=0) == 0 and run(T=0, x=None, ws=None) == 0
    assert run(T=129) == 6 and run(T=-1) == 1     # more tokens than the call takes
    assert run(k=0) == 1 and run(k=33) == 1 and run(E=0) == 1 and run(E=1025) == 1
    assert run(H=260) == 3 and run(I=4) == 1 and run(H=65536 + 8) == 1
    assert run(lim=-1.0) == 1 and run(lim=float("nan")) == 1
    assert run(n=need - 1) == 1 and run(ws=None) == 1
    for name in ("x", "ids", "w1", "w2", "out"):
        assert run(**{name: None}) == 1, name
    assert run(x=G + 8) == 3 and run(ids=G + 2) == 3 and run(w=G + 1) == 3 and run(err=G + 2) == 3

    def mx(fmt=1, sx=G, H=256, I=128, s1=G, s2=G):
        return lib.pgg_mx_moe_decode(fmt, G, sx, G, G, G, s1, G, s2, G, 4, 2, H, I, 8, 0.0, G, 1 << 30, None, None)
    assert mx(fmt=0) == 1 and mx(fmt=3) == 1
    assert mx(H=264) == 3 and mx(I=192) == 3      # whole 128-element atoms
    assert mx(sx=None) == 1 and mx(s1=None) == 1 and mx(sx=G + 2) == 3 and mx(s2=G + 8) == 3


def test_stall_hook_refusals(lib):
    def run(stall=0, wait=2_000_000):
        return lib.pgg_test_stalled_moe_decode(0, G, None, G, G, None, G, None, G, 4, 2, 256, 128, 8, stall, wait, G, 1 << 30,
                                               None, None)
    assert run(stall=-1) == 1 and run(wait=50_000) == 1 and run(wait=2_000_000_000) == 1


def test_binding_refuses_wrong_tensors():
    import precision_grouped_gemm_gb300 as pgg
    bf = torch.bfloat16
    x, g = torch.zeros(2, 64, dtype=bf), torch.zeros(64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        pgg.add_rmsnorm(x, None, g)
    with pytest.raises(ValueError, match="gamma"):
        pgg.add_rmsnorm(x, None, g.float())
    with pytest.raises(ValueError, match="residual"):
        pgg.add_rmsnorm(x, x[:1], g)
    with pytest.raises(ValueError, match="fmt"):
        pgg.add_rmsnorm(x, None, g, codes=torch.zeros(2, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="logits"):
        pgg.moe_route(torch.zeros(2, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="score"):
        pgg.moe_route(torch.zeros(2, 8), 2, score="tanh")
    with pytest.raises(ValueError, match="W1"):
        pgg.moe_decode(x, torch.zeros(2, 1, dtype=torch.int32), None, torch.zeros(3, 16, 64, dtype=bf),
                       torch.zeros(3, 64, 16, dtype=bf), ws=torch.zeros(16, dtype=torch.uint8))
