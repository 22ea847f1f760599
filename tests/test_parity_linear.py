"""GPU parity of the products with biases (grouped_linear) and of their gradient with the fp64 oracle.

Tolerances, from the arithmetic.  Z is a sum of K products and a bias in fp32: the tensor core adds
sixteen products at a time to the accumulator, each addition off by at most 2^-23 of the magnitudes
summed so far, so dz = (K / 16 + 16) 2^-23 mag.  An activation passes on dz times its slope, plus the
error of its own functions: 2^-18 of the value, and for gelu (z^2) 2^-23 of it, as erfc's argument is
rounded twice and erfc's relative slope is z^2.  A bf16 output adds half a step (2^-8), fp32 2^-24.
dZ has 2^-18 of |dY| times the terms that act' is made of; dbias the sums of those, and of n additions
in fp32 by eight warps (n / 8 + 32) 2^-24 of the magnitudes."""
import numpy as np
import pytest
import torch

from oracle import grouped_gemm as og
from oracle import linear as ol
import util

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FORMS = {None: {}, "silu": {"alpha": 1.702}, "gelu": {}, "swiglu": {"alpha": 1.702, "offset": 1.0, "limit": 1.5}}
HALF = {BF: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(BF)


def _np(t):
    return util.f64(t) if t.dtype == BF else t.detach().cpu().double().numpy()


def _near(got, ref, bound, what):
    g = _np(got)
    assert np.array_equal(np.isnan(g), np.isnan(ref)), f"{what}: other NaNs"
    with np.errstate(invalid="ignore"):
        err = np.where(np.isnan(ref) | (g == ref), 0.0, np.abs(g - ref))
    bad = ~(err <= np.where(np.isnan(ref), 1.0, bound + 1e-30))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(err / (bound + 1e-30)):.3g} of the bound"


def _split(rng, M, G, empty=()):
    w = rng.random(G) + 0.05
    w[list(empty)] = 0
    return rng.multinomial(M, w / w.sum()).astype(np.int32)


def _inputs(M, N, K, lens, seed, bias=True, residual=True, act=None, out=BF):
    rng = np.random.default_rng(seed)
    width = N // 2 if act == "swiglu" else N
    X, W = _bf(rng, M, K), _bf(rng, len(lens), N, K, scale=1.5 * K ** -0.5)
    b = _bf(rng, len(lens), N) if bias else None
    r = _bf(rng, M, width).to(out) if residual else None
    return X, W, b, r


def _dev(t):
    return None if t is None else t.to(DEV)


def _check(Y, Z, X, W, lens, b, r, act, form):
    """Y and Z against the oracle, row for row."""
    x, w = util.f64(X), util.f64(W)
    y0, z0, mag = ol.linear(x, w, lens, None if b is None else util.f64(b), None, act, **form)
    K = x.shape[1]
    dz = (K / 16 + 16) * 2.0 ** -23 * mag
    if Z is not None:
        _near(Z, z0, HALF[BF] * np.abs(z0) + dz, "Z")
    if act == "swiglu":
        one = np.ones_like(y0)
        slope = np.abs(ol.act_bwd(one, z0, act, **form))
        h = y0.shape[1]
        # the slope itself moves by less than its own terms over dz: twice it and a constant cover that
        dy = 2 * (slope[:, :h] * dz[:, :h] + slope[:, h:] * dz[:, h:]) + (dz[:, :h] + dz[:, h:]) * 2.0 ** -6
    elif act:
        dy = 1.3 * max(1.0, form.get("alpha", 1.0)) * dz  # |act'| <= 1.13 (gelu), 1.1 (silu, any alpha)
    else:
        dy = dz
    ref = y0 if r is None else y0 + _np(r)
    fn = (0.0 if act is None else 2.0 ** -18 * np.abs(y0) + (z0 ** 2 * 2.0 ** -23 * np.abs(y0) if act == "gelu" else 0.0))
    _near(Y, ref, HALF[Y.dtype] * np.abs(ref) + 2.0 ** -23 * (np.abs(y0) + np.abs(ref)) + dy + fn, "Y")


CASES = [  # M, N, K, G, empty groups
    (1, 8, 8, 1, ()), (1, 1024, 4096, 1, ()), (2, 264, 520, 1, ()), (37, 256, 4096, 1, ()), (130, 136, 64, 1, ()),
    (257, 272, 200, 1, ()), (600, 144, 328, 1, ()), (9, 128, 256, 5, (0, 4)), (64, 640, 192, 7, (2, 3)),
    (777, 400, 136, 3, (1,)), (1200, 128, 72, 64, (5, 63)), (300, 48, 1000, 200, tuple(range(0, 200, 7))),
    (1500, 1040, 264, 4, ()), (5000, 272, 128, 2, (0,))]


@pytest.mark.parametrize("act", list(FORMS))
@pytest.mark.parametrize("M,N,K,G,empty", CASES)
def test_linear(M, N, K, G, empty, act):
    N = N // 16 * 16 if act == "swiglu" else N
    N = max(N, 16) if act == "swiglu" else N
    rng = np.random.default_rng(M + N)
    lens = _split(rng, M, G, empty)
    out = torch.float32 if (M + K // 8) % 2 else BF
    X, W, b, r = _inputs(M, N, K, lens, N * K, act=act, out=out)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (X.to(DEV), W.to(DEV), None if G == 1 else torch.from_numpy(lens).to(DEV))
    Y, Z = pgg.grouped_linear(*args, bias=_dev(b), residual=_dev(r), act=act, save_z=True, out_dtype=out, err=err,
                              **FORMS[act])
    assert pgg.read_error(err) == 0
    _check(Y, Z, X, W, lens, b, r, act, FORMS[act])
    # without bias, residual and Z, and in the other type
    other = BF if out == torch.float32 else torch.float32
    Y, Z = pgg.grouped_linear(*args, act=act, out_dtype=other, **FORMS[act])
    assert Z is None
    _check(Y, None, X, W, lens, None, None, act, FORMS[act])
    again, _ = pgg.grouped_linear(*args, act=act, out_dtype=other, **FORMS[act])
    assert torch.equal(Y, again)


def test_linear_one_long_group_among_short_ones():
    # row tiles of very different fill: 1, 2, 15 .. 17, 31 .. 33, 127 .. 129, 255 .. 257, 511 .. 513 rows
    lens = np.array([1, 2, 0, 15, 16, 17, 31, 32, 33, 0, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1], dtype=np.int32)
    for act in FORMS:
        M, N, K = int(lens.sum()), 272, 136
        X, W, b, r = _inputs(M, N, K, lens, 5, act=act)
        Y, Z = pgg.grouped_linear(X.to(DEV), W.to(DEV), torch.from_numpy(lens).to(DEV), bias=_dev(b), residual=_dev(r),
                                  act=act, save_z=True, **FORMS[act])
        _check(Y, Z, X, W, lens, b, r, act, FORMS[act])


@pytest.mark.parametrize("act", list(FORMS))
@pytest.mark.parametrize("N,K,lens", [
    (2064, 328, [3000]), (1040, 520, [700]), (544, 1096, [1, 2, 0, 15, 16, 17, 33, 65, 97, 129, 193, 257, 0, 385, 513]),
    (4112, 200, [150] * 16), (4112, 200, [1030, 0, 22])])
def test_linear_fp32_in_tiles_of_every_height(N, K, lens, act):
    # long and short groups, whose rows are shared out evenly over their tiles; the residual in place
    lens = np.array(lens, dtype=np.int32)
    M, width = int(lens.sum()), N // 2 if act == "swiglu" else N
    X, W, b, r = _inputs(M, N, K, lens, N + K, act=act, out=torch.float32)
    buf = torch.full((M + 9, width), 7.0, device=DEV)
    buf[:M] = r.to(DEV)
    gl = None if len(lens) == 1 else torch.from_numpy(lens).to(DEV)
    Y, Z = pgg.grouped_linear(X.to(DEV), W.to(DEV), gl, bias=_dev(b), residual=buf[:M], Y=buf[:M], act=act, save_z=True,
                              **FORMS[act])
    assert (buf[M:] == 7).all()
    _check(Y, Z, X, W, lens, b, r, act, FORMS[act])


def test_linear_equals_the_swiglu_layer():
    lens = np.array([70, 0, 200, 33], dtype=np.int32)
    X, W, _, _ = _inputs(303, 256, 192, lens, 9, act="swiglu")
    gl = torch.from_numpy(lens).to(DEV)
    A, H = pgg.grouped_fc1_swiglu(X.to(DEV), W.to(DEV), gl, swiglu_limit=1.0)
    Y, Z = pgg.grouped_linear(X.to(DEV), W.to(DEV), gl, act="swiglu", limit=1.0, save_z=True)
    util.assert_close(Y, util.f64(A), "A", rel=2 ** -7, abs_rms=1e-5)
    util.assert_close(Z, util.f64(H), "H", rel=2 ** -7, abs_rms=1e-5)


@pytest.mark.parametrize("M,G", [(40, 1), (40, 3), (700, 1), (700, 3)])
def test_linear_special_values_stay_in_their_rows_and_columns(M, G):
    rng = np.random.default_rng(M)
    lens = _split(rng, M, G)
    N, K = 272, 200
    X, W, b, r = _inputs(M, N, K, lens, 7)
    X[3, 5], X[M - 1, 0] = float("nan"), float("inf")
    W[0, 17, 9] = float("nan")
    b[G - 1, 30] = float("-inf")
    r[5, 40] = float("nan")
    Y, _ = pgg.grouped_linear(X.to(DEV), W.to(DEV), torch.from_numpy(lens).to(DEV), bias=_dev(b), residual=_dev(r))
    got = _np(Y)
    clean = np.ones((M, N), bool)
    clean[[3, M - 1]] = False
    clean[:lens[0], 17] = False
    clean[M - lens[-1]:, 30] = False
    clean[5, 40] = False
    assert np.isnan(got[3]).all() and np.isnan(got[:lens[0], 17]).all() and np.isnan(got[5, 40])
    last = got[M - lens[-1]:, 30]
    keep = ~np.isin(np.arange(M - lens[-1], M), [3, M - 1])
    assert (last[keep] == -np.inf).all()
    assert not np.isfinite(got[M - 1]).any()
    assert np.isfinite(got[clean]).all()


def test_linear_keeps_a_nan_through_the_clamps():
    X = torch.zeros(2, 64, dtype=BF, device=DEV)
    X[0, 0] = float("nan")
    W = torch.ones(32, 64, dtype=BF, device=DEV)
    Y, _ = pgg.grouped_linear(X, W, act="swiglu", limit=1.0)
    assert torch.isnan(Y[0]).all() and (Y[1] == 0).all()


def test_linear_residual_in_place_and_rows_behind():
    rng = np.random.default_rng(4)
    for M, G in ((5, 1), (333, 1), (333, 4)):
        lens = _split(rng, M, G)
        for out in (BF, torch.float32):
            X, W, b, r = _inputs(M, 136, 72, lens, M, out=out)
            buf = torch.full((M + 40, 136), 7.0, dtype=out, device=DEV)
            buf[:M] = r.to(DEV)
            gl = torch.from_numpy(lens).to(DEV)
            Y, _ = pgg.grouped_linear(X.to(DEV), W.to(DEV), gl, bias=_dev(b), residual=buf[:M], Y=buf[:M])
            ref, _ = pgg.grouped_linear(X.to(DEV), W.to(DEV), gl, bias=_dev(b), residual=_dev(r), out_dtype=out)
            assert torch.equal(Y, ref) and (buf[M:] == 7).all()


@pytest.mark.parametrize("lens", [[5, -1, 6], [5, 4, 2], [5, 4, 0], [2 ** 31 - 1, 2 ** 31 - 1, 12]])
@pytest.mark.parametrize("M,act", [(10, None), (10, "swiglu"), (800, None), (800, "swiglu")])
def test_linear_bad_lens_write_nothing(lens, M, act):
    lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    X, W = torch.ones(M, 64, dtype=BF, device=DEV), torch.ones(3, 64, 64, dtype=BF, device=DEV)
    Y = torch.full((M, 32 if act else 64), 3.0, dtype=BF, device=DEV)
    Z = torch.full((M, 64), 3.0, dtype=BF, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pgg.grouped_linear(X, W, lens, act=act, Y=Y, Z=Z, err=err)
    assert pgg.read_error(err) == 16 and (Y == 3).all() and (Z == 3).all()
    db = torch.full((3, 64), 3.0, device=DEV)
    dz = torch.full((M, 64), 3.0, dtype=BF, device=DEV)
    err.zero_()
    pgg.grouped_linear_bwd(Y, Z if act else None, lens, act=act, dZ=dz if act else None, dbias=db, err=err)
    assert pgg.read_error(err) == 16 and (db == 3).all() and (dz == 3).all()


def test_linear_empty_batch():
    X, W = torch.ones(0, 64, dtype=BF, device=DEV), torch.ones(3, 64, 64, dtype=BF, device=DEV)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    Y, Z = pgg.grouped_linear(X, W, lens, save_z=True)
    assert Y.shape == (0, 64) and Z.shape == (0, 64)
    dz, db = pgg.grouped_linear_bwd(Y, Z, lens, act="silu")
    assert dz.shape == (0, 64) and db.shape == (3, 64) and (db == 0).all()


@pytest.mark.parametrize("act", list(FORMS))
@pytest.mark.parametrize("M,N,G,empty", [(1, 8, 1, ()), (33, 1032, 1, ()), (777, 1040, 5, (3,)), (4100, 272, 3, (0,)),
                                         (300, 64, 257, tuple(range(0, 257, 3))), (2000, 4112, 2, ()), (70, 16, 1, ()),
                                         (1500, 528, 1024, tuple(range(1, 1024, 2)))])
def test_linear_bwd(M, N, G, empty, act):
    N = (N + 15) // 16 * 16 if act == "swiglu" else N
    rng = np.random.default_rng(M + N)
    lens = _split(rng, M, G, empty)
    Z, dY = _bf(rng, M, N, scale=1.5), _bf(rng, M, N // 2 if act == "swiglu" else N)
    gl = None if G == 1 else torch.from_numpy(lens).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    run = lambda **kw: pgg.grouped_linear_bwd(dY.to(DEV), Z.to(DEV) if act else None, gl, act=act, err=err,  # noqa: E731
                                              **FORMS[act], **kw)
    dz, db = run()
    assert pgg.read_error(err) == 0
    z, dy = util.f64(Z), util.f64(dY)
    rz, rb, _ = ol.linear_bwd(dy, z, lens, act, **FORMS[act])
    form = FORMS[act]
    if act == "swiglu":
        g, u = np.split(z, 2, axis=1)
        g, u = np.minimum(g, form["limit"]), np.clip(u, -form["limit"], form["limit"])
        terms = np.concatenate([np.abs(dy) * np.abs(u + form["offset"]) * (1 + np.abs(form["alpha"] * g)),
                                np.abs(dy) * np.abs(g)], axis=1)
    else:
        terms = np.abs(dy) * (1 + 2 * np.abs(z)) if act else np.abs(dy)
    fn = 0.0 if act is None else 2.0 ** -18
    _near(dz, rz, (HALF[BF] if act else 0.0) * np.abs(rz) + fn * terms, "dZ")
    ends = np.concatenate([[0], np.cumsum(lens)])
    mag = np.array([terms[ends[i]:ends[i + 1]].sum(0) for i in range(G)])
    _near(db, rb, (fn + (lens[:, None] / 8 + 32) * 2.0 ** -24) * mag, "dbias")
    ws = torch.full((pgg.grouped_linear_bwd_workspace_size(M, N, G, act) + 64,), 255, dtype=torch.uint8, device=DEV)
    dz2, db2 = run(ws=ws)   # whatever the workspace holds, and the same bits again
    assert torch.equal(dz, dz2) and torch.equal(db, db2)
    if act:
        buf = Z.to(DEV)
        pgg.grouped_linear_bwd(dY.to(DEV), buf, gl, act=act, dZ=buf, **FORMS[act])
        assert torch.equal(buf, dz)


@pytest.mark.parametrize("act", [None, "silu", "swiglu"])
@pytest.mark.parametrize("lens", [[1] * 70, [0] * 31 + [3, 0, 9, 8, 7, 1, 600, 0, 2, 40] + [1, 2, 0] * 20 + [33] + [0] * 30,
                                  [5000] + [0, 1, 12] * 80, [2] * 1024])
def test_linear_bwd_of_groups_with_few_rows(lens, act):
    # groups inside a run, over the ends of runs and over many of them; empty ones before, between and behind
    lens = np.array(lens, dtype=np.int32)
    M, N, form = int(lens.sum()), 528, FORMS[act]
    rng = np.random.default_rng(M)
    Z, dY = _bf(rng, M, N, scale=1.5), _bf(rng, M, N // 2 if act == "swiglu" else N)
    dz, db = pgg.grouped_linear_bwd(dY.to(DEV), Z.to(DEV) if act else None, torch.from_numpy(lens).to(DEV), act=act, **form)
    one, rb1 = pgg.grouped_linear_bwd(dY.to(DEV), Z.to(DEV) if act else None, None, act=act, **form)
    assert torch.equal(dz, one)  # (an element's gradient is its own; test_linear_bwd checks it)
    rz, rb, _ = ol.linear_bwd(util.f64(dY), util.f64(Z), lens, act, **form)
    # dZ's own error, 2^-18 of its terms: |dY| (1 + 1.7 |g|) (|u| + 1) <= 11 |dY| for |g|, |u| <= 1.5, or 1 + 2 |z|
    dy = np.abs(util.f64(dY))
    terms = np.tile(11 * dy, 2) if act == "swiglu" else dy * (1 + 2 * np.abs(util.f64(Z))) if act else dy
    ends = np.concatenate([[0], np.cumsum(lens)])
    mag = np.array([terms[ends[i]:ends[i + 1]].sum(0) for i in range(len(lens))])
    _near(db, rb, ((2.0 ** -18 if act else 0.0) + (lens[:, None] / 8 + 32) * 2.0 ** -24) * mag, "dbias")


def test_linear_gradients_by_differences_through_the_framework():
    """dX, dW, dbias and the residual's gradient from the calls that a training step makes, against
    central differences of the fp64 oracle along random directions."""
    rng = np.random.default_rng(11)
    lens = np.array([40, 0, 25], dtype=np.int32)
    M, N, K = 65, 96, 64
    for act, form in FORMS.items():
        X, W, b, r = _inputs(M, N, K, lens, 3, act=act)
        dY = _bf(rng, M, r.shape[1])
        gl = torch.from_numpy(lens).to(DEV)
        Y, Z = pgg.grouped_linear(X.to(DEV), W.to(DEV), gl, bias=_dev(b), residual=_dev(r), act=act, save_z=True, **form)
        dz, db = pgg.grouped_linear_bwd(dY.to(DEV), Z if act else None, gl, act=act, **form)
        g = {"X": pgg.grouped_gemm_dgrad(dz, W.to(DEV), gl), "W": pgg.grouped_gemm_wgrad(X.to(DEV), dz, gl), "b": db}
        v = {"X": util.f64(X), "W": util.f64(W), "b": util.f64(b)}
        f = lambda v: np.sum(ol.linear(v["X"], v["W"], lens, v["b"], util.f64(r), act, **form)[0] * util.f64(dY))  # noqa: E731
        for name, got in g.items():
            got = got.double().cpu().numpy().reshape(v[name].shape)
            d = np.sign(got) * np.abs(rng.standard_normal(got.shape))  # every term adds up
            up, dn = dict(v), dict(v)
            up[name], dn[name] = v[name] + 1e-5 * d, v[name] - 1e-5 * d
            assert np.sum(got * d) == pytest.approx((f(up) - f(dn)) / 2e-5, rel=1e-2), (act, name)


def test_linear_on_another_stream_and_in_a_graph():
    lens = np.array([30, 0, 99], dtype=np.int32)
    X, W, b, r = (_dev(t) for t in _inputs(129, 256, 192, lens, 13))
    gl = torch.from_numpy(lens).to(DEV)
    ref, refz = pgg.grouped_linear(X, W, gl, bias=b, residual=r, act="silu", save_z=True)
    rdz, rdb = pgg.grouped_linear_bwd(ref, refz, gl, act="silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y, Z = pgg.grouped_linear(X, W, gl, bias=b, residual=r, act="silu", save_z=True, stream=s)
    dz, db = pgg.grouped_linear_bwd(Y, Z, gl, act="silu", stream=s)
    s.synchronize()
    assert torch.equal(Y, ref) and torch.equal(dz, rdz) and torch.equal(db, rdb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y, Z = pgg.grouped_linear(X, W, gl, bias=b, residual=r, act="silu", save_z=True)
        dz, db = pgg.grouped_linear_bwd(Y, Z, gl, act="silu")
    x2 = _bf(np.random.default_rng(5), 129, 192).to(DEV)
    for x in (X.clone(), x2):
        X.copy_(x)
        g.replay()
        ref, refz = pgg.grouped_linear(x, W, gl, bias=b, residual=r, act="silu", save_z=True)
        rdz, rdb = pgg.grouped_linear_bwd(ref, refz, gl, act="silu")
        assert torch.equal(Y, ref) and torch.equal(dz, rdz) and torch.equal(db, rdb)


def test_linear_offsets_past_32_bits():
    # W of 2^31 elements and more: the named groups lie at both ends
    G, N, K = 260, 4096, 2048
    W = torch.zeros(G, N, K, dtype=BF, device=DEV)
    lens = torch.zeros(G, dtype=torch.int32, device=DEV)
    lens[0], lens[-1] = 3, 5
    rng = np.random.default_rng(1)
    X, w0, w1 = _bf(rng, 8, K), _bf(rng, N, K, scale=0.02), _bf(rng, N, K, scale=0.02)
    W[0], W[-1] = w0.to(DEV), w1.to(DEV)
    Y, _ = pgg.grouped_linear(X.to(DEV), W, lens)
    ref = np.concatenate([util.f64(X)[:3] @ util.f64(w0).T, util.f64(X)[3:] @ util.f64(w1).T])
    mag = np.concatenate([np.abs(util.f64(X))[:3] @ np.abs(util.f64(w0)).T, np.abs(util.f64(X))[3:] @ np.abs(util.f64(w1)).T])
    _near(Y, ref, HALF[BF] * np.abs(ref) + (K / 16 + 16) * 2.0 ** -23 * mag, "Y")


@pytest.mark.parametrize("M,N,K,G,act", [(600, 512, 512, 2, 0), (600, 512, 512, 2, 3), (12, 512, 512, 2, 0),
                                         (12, 512, 1024, 1, 0), (12, 512, 1024, 1, 3), (4000, 2048, 512, 1, 0)])
@pytest.mark.parametrize("stall_at", [0, 3])
def test_linear_wait_expiry(M, N, K, G, act, stall_at):
    """Loads that stop: the kernel gives up within its limit, says so, and the next call is right."""
    X, W = torch.ones(M, K, dtype=BF, device=DEV), torch.ones(G, N, K, dtype=BF, device=DEV)
    lens = torch.full((G,), M // G, dtype=torch.int32, device=DEV)
    Y = torch.zeros(M, N // 2 if act == 3 else N, dtype=BF, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    st = pgg.lib().pgg_test_stalled_linear(X.data_ptr(), W.data_ptr(), lens.data_ptr(), Y.data_ptr(), M, N, K, G, act,
                                           stall_at, 2_000_000, err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0 and pgg.read_error(err) == 17
    err.zero_()
    Y, _ = pgg.grouped_linear(X, W, lens, act="swiglu" if act else None, err=err)
    assert pgg.read_error(err) == 0
    want = float(og.swiglu_fwd(np.full((1, 2), float(K)))[0, 0]) if act else float(K)
    assert (Y.float() == torch.tensor(want).to(BF).float().item()).all()


@pytest.mark.parametrize("act", list(FORMS))
@pytest.mark.parametrize("lens", [[1100, 0, 515, 2000], [513, 700], [4096 + 17]])
def test_linear_long_groups(lens, act):
    # groups of several row tiles, ragged at their ends; column tiles that end inside a CTA pair's columns
    lens = np.array(lens, dtype=np.int32)
    for N, K in ((336, 200), (176, 72), (1296, 64)):
        X, W, b, r = _inputs(int(lens.sum()), N, K, lens, N, act=act)
        Y, Z = pgg.grouped_linear(X.to(DEV), W.to(DEV), torch.from_numpy(lens).to(DEV), bias=_dev(b), residual=_dev(r),
                                  act=act, save_z=True, **FORMS[act])
        _check(Y, Z, X, W, lens, b, r, act, FORMS[act])
        again, z2 = pgg.grouped_linear(X.to(DEV), W.to(DEV), torch.from_numpy(lens).to(DEV), bias=_dev(b), residual=_dev(r),
                                       act=act, save_z=True, **FORMS[act])
        assert torch.equal(Y, again) and torch.equal(Z, z2)


def test_tensors_of_another_device_are_refused(monkeypatch):
    from precision_grouped_gemm_gb300 import _binding
    x, w = torch.ones(2, 64, dtype=BF, device=DEV), torch.ones(32, 64, dtype=BF, device=DEV)
    pgg.grouped_linear(x, w)
    monkeypatch.setattr(_binding, "_raw_device", lambda: 1)   # as if another device were the current one
    for call in (lambda: pgg.grouped_linear(x, w), lambda: pgg.grouped_linear_bwd(x), lambda: pgg.block_join(x, x),
                 lambda: pgg.block_join_bwd(None, x, x)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_linear_on_four_streams_at_once():
    # calls of every kernel (few rows, short and long groups, both types) that overlap
    cases = []
    for i, (M, N, K, G, act, out) in enumerate([(1, 2048, 2048, 1, None, BF), (40, 1024, 2048, 1, "swiglu", BF),
                                                (700, 512, 512, 5, "gelu", BF), (3000, 1024, 512, 2, "swiglu", BF),
                                                (37, 256, 2048, 1, None, torch.float32), (900, 512, 512, 3, "silu", torch.float32)]):
        lens = _split(np.random.default_rng(i), M, G)
        X, W, b, r = (_dev(t) for t in _inputs(M, N, K, lens, i, act=act, out=out))
        gl = torch.from_numpy(lens).to(DEV)
        kw = dict(bias=b, residual=r, act=act, out_dtype=out, **FORMS[act])
        cases.append((X, W, gl, kw, pgg.grouped_linear(X, W, gl, **kw)[0]))
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for n in range(30):
        for j, s in enumerate(streams):
            X, W, gl, kw, ref = cases[(n + j) % len(cases)]
            with torch.cuda.stream(s):
                got.append((pgg.grouped_linear(X, W, gl, **kw)[0], ref))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
