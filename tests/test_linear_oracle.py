"""CPU pins of the oracle of the products with biases and of the joints between blocks, and the
refusals of their entry points (argument checks run before any CUDA call)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import linear as ol

KINDS = [(None, {}), ("silu", {"alpha": 1.702}), ("gelu", {}), ("swiglu", {"alpha": 1.702, "offset": 1.0, "limit": 1.2}),
         ("swiglu", {})]


def test_philox_known_answers():
    # the published generator's test vectors
    assert ol.philox4x32((0,) * 4, (0,) * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ol.philox4x32((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ol.philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_keep_is_a_share_of_p_and_follows_seed_and_offset():
    m = ol.keep(40, 100, 0.25, (7, 3))
    assert abs(m.mean() - 0.75) < 5 * math.sqrt(0.25 * 0.75 / m.size)
    assert (m != ol.keep(40, 100, 0.25, (8, 3))).any() and (m != ol.keep(40, 100, 0.25, (7, 4))).any()
    np.testing.assert_array_equal(m[:10], ol.keep(10, 100, 0.25, (7, 3)))  # the tensor's first rows
    np.testing.assert_array_equal(ol.keep(3, 8, 0.5, (-1, -2)), ol.keep(3, 8, 0.5, (2 ** 64 - 1, 2 ** 64 - 2)))


@pytest.mark.parametrize("kind,form", KINDS)
def test_linear_by_loops(kind, form):
    r = np.random.default_rng(1)
    lens, N, K = [2, 0, 3], 6, 4
    X, W, b = r.standard_normal((5, K)), r.standard_normal((3, N, K)), r.standard_normal((3, N))
    res = r.standard_normal((5, N // 2 if kind == "swiglu" else N))
    Y, Z, _ = ol.linear(X, W, lens, b, res, kind, **form)
    owner = [0, 0, 2, 2, 2]
    a, off, lim = form.get("alpha", 1.0), form.get("offset", 0.0), form.get("limit", 0.0)
    for m in range(5):
        z = [b[owner[m], n] + sum(X[m, k] * W[owner[m], n, k] for k in range(K)) for n in range(N)]
        np.testing.assert_allclose(Z[m], z, rtol=1e-12)
        for n in range(res.shape[1]):
            if kind == "swiglu":
                g, u = z[n], z[n + 3]
                if lim:
                    g, u = min(g, lim), max(-lim, min(u, lim))
                y = g / (1 + math.exp(-a * g)) * (u + off)
            else:
                y = {None: z[n], "silu": z[n] / (1 + math.exp(-a * z[n])),
                     "gelu": z[n] * 0.5 * (1 + math.erf(z[n] / 2 ** 0.5))}[kind]
            assert Y[m, n] == pytest.approx(y + res[m, n], rel=1e-12)


@pytest.mark.parametrize("kind,form", KINDS)
def test_linear_bwd_by_differences(kind, form):
    r = np.random.default_rng(2)
    Z = r.standard_normal((6, 8))
    dY = r.standard_normal((6, 4 if kind == "swiglu" else 8))
    dZ, db, _ = ol.linear_bwd(dY, Z, [4, 0, 2], kind, **form)
    e = 1e-6
    for i in range(6):
        for j in range(8):
            up, dn = Z.copy(), Z.copy()
            up[i, j] += e
            dn[i, j] -= e
            num = np.sum(dY * (ol.act(up, kind, **form) - ol.act(dn, kind, **form))) / (2 * e)
            assert dZ[i, j] == pytest.approx(num, rel=1e-6, abs=1e-8)
    np.testing.assert_allclose(db, [dZ[:4].sum(0), np.zeros(8), dZ[4:].sum(0)], rtol=1e-12)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "row", "column"])
def test_join_bwd_by_differences(post, gate):
    r = np.random.default_rng(3)
    R, C, p, ra, rb, eps = 3, 8, 0.3, 0.9, 0.5, 1e-5
    v = {"x": r.standard_normal((R, C)), "residual": r.standard_normal((R, C)), "gamma": r.standard_normal(C),
         "gamma_post": r.standard_normal(C) if post else None,
         "gate": {None: None, "row": r.standard_normal((R, 1)), "column": r.standard_normal(C)}[gate]}
    mask = ol.keep(R, C, p, (5, 6))
    dy, dh = r.standard_normal((R, C)), r.standard_normal((R, C))
    run = lambda v: ol.join(v["x"], v["residual"], v["gamma_post"], v["gamma"], v["gate"], ra, rb, p, mask, eps)  # noqa: E731
    s, y, r1, r2 = run(v)
    t = v["x"] / np.sqrt(np.mean(v["x"] ** 2, 1, keepdims=True) + eps) * v["gamma_post"] if post else v["x"]
    np.testing.assert_allclose(s, ra * v["residual"] + rb * (1 if gate is None else v["gate"]) * t * mask / 0.7, rtol=1e-12)
    np.testing.assert_allclose(y, s / np.sqrt(np.mean(s * s, 1, keepdims=True) + eps) * v["gamma"], rtol=1e-12)
    g = ol.join_bwd(dy, dh, v["x"], s, r1, r2, v["gamma_post"], v["gamma"], v["gate"], ra, rb, p, mask)
    for name, value in v.items():
        if value is None:
            continue
        got = g["d" + name].reshape(value.shape)
        for i in np.ndindex(value.shape):
            e = 1e-6
            up, dn = dict(v), dict(v)
            up[name], dn[name] = value.copy(), value.copy()
            up[name][i] += e
            dn[name][i] -= e
            loss = lambda w: (lambda o: np.sum(o[0] * dh) + np.sum(o[1] * dy))(run(w))  # noqa: E731
            assert got[i] == pytest.approx((loss(up) - loss(dn)) / (2 * e), rel=1e-5, abs=1e-7), (name, i)


# ---------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    from precision_grouped_gemm_gb300 import _binding, build
    build.build()
    return _binding.lib()


P = 1 << 20  # an aligned address that is never followed
NAN, INF = float("nan"), float("inf")


def test_linear_refusals(lib):
    def run(X=P, W=P, lens=P, bias=P, res=P, Y=P, dt=1, Z=P, M=8, N=64, K=64, G=2, act=0, alpha=1.0, off=0.0, lim=0.0,
            err=None):
        return lib.pgg_grouped_linear(X, W, lens, bias, res, Y, dt, Z, M, N, K, G, act, alpha, off, lim, err, None)
    assert run(M=0) == 0 and run(M=0, X=None, Y=None) == 0
    assert run(X=None) == 1 and run(W=None) == 1 and run(Y=None) == 1
    assert run(M=-1) == 1 and run(M=1 << 31) == 1 and run(G=0) == 1 and run(G=1025) == 1
    assert run(lens=None) == 1                      # several groups need their lengths
    assert run(N=4) == 1 and run(K=0) == 1 and run(N=68) == 3 and run(K=12) == 3
    assert run(N=72, act=3) == 3                    # halves of whole 16-byte pieces
    assert run(act=4) == 1 and run(act=-1) == 1 and run(dt=2) == 1
    for bad in (NAN, INF, -INF):
        assert run(alpha=bad) == 1 and run(off=bad) == 1 and run(lim=bad) == 1
    assert run(lim=-1.0) == 1
    for name in ("X", "W", "bias", "res", "Y", "Z"):
        assert run(**{name: P + 8}) == 3, name
    assert run(lens=P + 2) == 3 and run(err=P + 1) == 3

    def stall(at=0, ns=2_000_000):
        return lib.pgg_test_stalled_linear(P, P, P, P, 8, 64, 64, 2, 0, at, ns, None, None)
    assert stall(at=-1) == 1 and stall(ns=50_000) == 1 and stall(ns=2_000_000_000) == 1


def test_linear_bwd_refusals(lib):
    size = ctypes.c_size_t(0)
    assert lib.pgg_grouped_linear_bwd_workspace_size(100, 64, 3, 1, ctypes.byref(size)) == 0
    need = size.value
    assert lib.pgg_grouped_linear_bwd_workspace_size(100, 60, 3, 1, ctypes.byref(size)) == 3
    assert lib.pgg_grouped_linear_bwd_workspace_size(100, 72, 3, 3, ctypes.byref(size)) == 3
    assert lib.pgg_grouped_linear_bwd_workspace_size(100, 64, 3, 1, None) == 1

    def run(dY=P, Z=P, lens=P, dZ=P, db=P, M=100, N=64, G=3, act=1, alpha=1.0, off=0.0, lim=0.0, ws=P, n=need, err=None):
        return lib.pgg_grouped_linear_bwd(dY, Z, lens, dZ, db, M, N, G, act, alpha, off, lim, ws, n, err, None)
    assert run(dY=None) == 1 and run(Z=None) == 1 and run(db=None) == 1 and run(ws=None) == 1 and run(n=need - 1) == 1
    assert run(act=0) == 1 and run(act=0, Z=None) == 1     # Z and dZ belong to an activation
    assert run(lens=None) == 1 and run(G=0) == 1 and run(M=-1) == 1 and run(act=4) == 1
    assert run(lim=-1.0) == 1 and run(alpha=NAN) == 1 and run(off=INF) == 1
    for name in ("dY", "Z", "dZ", "db", "ws"):
        assert run(**{name: P + 8}) == 3, name
    assert run(lens=P + 2) == 3 and run(err=P + 2) == 3


def test_join_refusals(lib):
    def run(x=P, r=P, g1=P, g2=P, gate=None, kind=0, rng=None, R=4, C=64, p=0.0, ra=1.0, rb=1.0, eps=1e-6, fmt=1, h=P, y=P,
            c=P, s=P, q1=P, q2=P):
        return lib.pgg_block_join(x, r, g1, g2, gate, kind, rng, R, C, p, ra, rb, eps, fmt, h, y, c, s, q1, q2, None)
    assert run(R=0) == 0
    assert run(x=None) == 1 and run(R=-1) == 1 and run(C=0) == 1 and run(C=16384 + 32) == 1 and run(C=72) == 3
    assert run(fmt=7) == 1 and run(fmt=0) == 1 and run(s=None) == 1 and run(c=None) == 1
    assert run(g2=None) == 1                                # y, codes and rstd belong to gamma
    assert run(g1=None) == 1                                # rstd_post to gamma_post
    assert run(gate=P) == 1 and run(kind=1) == 1 and run(kind=3, gate=P) == 1
    assert run(p=0.1) == 1                                  # no generator state
    assert run(p=1.0, rng=P) == 1 and run(p=-0.1, rng=P) == 1 and run(p=NAN, rng=P) == 1
    assert run(ra=NAN) == 1 and run(rb=INF) == 1 and run(eps=-1.0) == 1 and run(eps=NAN) == 1
    assert run(fmt=0, h=None, y=None, c=None, s=None, q1=None, q2=None) == 1
    for name in ("x", "r", "g1", "g2", "h", "y", "c"):
        assert run(**{name: P + 8}) == 3, name
    assert run(q1=P + 2) == 3 and run(q2=P + 2) == 3 and run(gate=P + 8, kind=2) == 3 and run(gate=P + 2, kind=1) == 3
    assert run(rng=P + 4, p=0.1) == 3


def test_join_bwd_refusals(lib):
    size = ctypes.c_size_t(0)
    assert lib.pgg_block_join_bwd_workspace_size(10, 64, ctypes.byref(size)) == 0 and size.value >= 10 * 64 * 12
    need = size.value
    assert lib.pgg_block_join_bwd_workspace_size(10, 60, ctypes.byref(size)) == 3

    def run(dy=P, dh=P, x=P, h=P, q1=P, q2=P, g1=P, g2=P, gate=P, kind=1, rng=None, R=10, C=64, p=0.0, ra=1.0, rb=1.0,
            dx=P, dr=P, d1=P, d2=P, dg=P, ws=P, n=need):
        return lib.pgg_block_join_bwd(dy, dh, x, h, q1, q2, g1, g2, gate, kind, rng, R, C, p, ra, rb, dx, dr, d1, d2, dg, ws,
                                      n, None)
    for name in ("dy", "x", "h", "q1", "q2", "dx", "d1", "d2", "dg", "ws", "g1", "g2"):
        assert run(**{name: None}) == 1, name
    assert run(gate=None) == 1 and run(gate=None, kind=0) == 1 and run(p=0.5) == 1 and run(n=need - 1) == 1
    for name in ("dy", "dh", "x", "h", "g1", "g2", "dx", "dr", "ws"):
        assert run(**{name: P + 8}) == 3, name
    assert run(q1=P + 2) == 3 and run(d1=P + 2) == 3 and run(dg=P + 1) == 3 and run(C=12) == 3 and run(kind=5) == 1


def test_binding_refuses_wrong_tensors():
    import precision_grouped_gemm_gb300 as pgg
    bf = torch.bfloat16
    x, w, g = torch.zeros(2, 64, dtype=bf), torch.zeros(3, 32, 64, dtype=bf), torch.zeros(64, dtype=bf)
    lens = torch.zeros(3, dtype=torch.int32)
    for match, args, kw in [
            ("CUDA", (x, w, lens), {}), ("W", (x, w[:, :, :32], lens), {}), ("group_lens", (x, w), {}),
            ("group_lens", (x, w, lens[:2]), {}), ("group_lens", (x, w, lens.long()), {}), ("act", (x, w, lens), {"act": "tanh"}),
            ("bias", (x, w, lens), {"bias": g}), ("residual", (x, w, lens), {"residual": x}),
            ("residual", (x, w, lens), {"residual": torch.zeros(2, 32, dtype=bf), "out_dtype": torch.float32}),
            ("Y must", (x, w, lens), {"out_dtype": torch.float16})]:
        with pytest.raises(ValueError, match=match):
            pgg.grouped_linear(*args, **kw)
    for match, args, kw in [("act needs Z", (x,), {"act": "silu"}), ("need act", (x, x), {}),
                            ("Z must", (x, x), {"act": "swiglu"})]:
        with pytest.raises(ValueError, match=match):
            pgg.grouped_linear_bwd(*args, **kw)
    for match, kw in [("gate", {"gate": torch.zeros(3)}), ("gate", {"gate": g[:8]}), ("rng", {"p": 0.5}), ("p must", {"p": 1.0}),
                      ("gamma", {"fmt": "e4m3"}), ("rstd_post", {"rstd_post": torch.zeros(2)}),
                      ("rng", {"p": 0.5, "rng": torch.zeros(2)}), ("fmt", {"gamma": g, "codes": x})]:
        with pytest.raises(ValueError, match=match):
            pgg.block_join(x, x, **kw)
    for match, kw in [("dy needs", {"dy": x}), ("gamma needs", {"gamma": g}), ("rstd_post", {"gamma_post": g}),
                      ("dgate", {"dgate": torch.zeros(2)})]:
        with pytest.raises(ValueError, match=match):
            pgg.block_join_bwd(kw.pop("dy", None), x, x, **kw)
