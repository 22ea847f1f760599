"""GPU parity of the joint between two blocks (norms, gate, dropout, scaled residual) with the fp64 oracle.

Tolerances, from the arithmetic: every value is computed in fp32 by a few dozen operations from the
inputs, sums over at most 16384 columns in a tree, so 2^-18 of the magnitudes that a value is made of;
a bf16 output adds half a step, 2^-8 of itself.  Dropout's mask is exact.  MX codes come from an fp32
value that may sit on the other side of a rounding boundary than the fp64 one: at most one code in a
thousand may differ, by one step of the grid."""
import numpy as np
import pytest
import torch

from oracle import linear as ol
from oracle import mx as omx
import util

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(BF)


def _np(t):
    return util.f64(t) if t.dtype == BF else t.detach().cpu().double().numpy()


def _near(got, ref, mag, what):
    g = _np(got).reshape(np.shape(ref))
    bound = (2.0 ** -8 if got.dtype == BF else 0.0) * np.abs(ref) + 2.0 ** -18 * mag + 1e-30
    err = np.abs(g - ref)
    assert (err <= bound).all(), f"{what}: {(~(err <= bound)).sum()} of {err.size}, worst {np.nanmax(err / bound):.3g} of the bound"


def _check_codes(codes, scales, y, fmt):
    R, C = y.shape
    rs, rc = omx.quantize_blocks(fmt, y.reshape(R, C // 32, 32))
    gs, gc = scales.cpu().numpy(), codes.cpu().numpy()
    gc = (omx.unpack_e2m1(gc) if fmt == "e2m1" else gc).reshape(R, C // 32, 32)
    assert np.mean(gs != rs) <= 1e-3
    same = gs == rs
    a, b = gc[same].astype(int), rc[same].astype(int)
    assert np.mean(a != b) <= 1e-3 and np.abs(a - b).max(initial=0) <= 1


def _case(R, C, post, gate, p, fmt, seed, residual=True):
    rng = np.random.default_rng(seed)
    t = {"x": _bf(rng, R, C), "residual": _bf(rng, R, C, scale=3.0) if residual else None,
         "gamma_post": _bf(rng, C) if post else None, "gamma": _bf(rng, C),
         "gate": {None: None, "token": torch.from_numpy(rng.standard_normal(R).astype(np.float32)),
                  "channel": _bf(rng, C)}[gate],
         "rng": torch.from_numpy(rng.integers(-2 ** 63, 2 ** 63 - 1, 2)) if p else None}
    d = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    g64 = None if gate is None else _np(t["gate"])[:, None] if gate == "token" else _np(t["gate"])
    mask = ol.keep(R, C, p, t["rng"].tolist() if p else None)
    n = {k: None if t[k] is None else _np(t[k]) for k in ("x", "residual", "gamma_post", "gamma")}
    return t, d, n, g64, mask


CASES = [  # R, C, post norm, gate, p, fmt
    (1, 32, True, None, 0.0, "e4m3"), (4, 4096, True, "token", 0.0, "e4m3"), (3, 96, False, "channel", 0.5, "e2m1"),
    (5, 1056, True, "channel", 0.1, None), (7, 8, True, "token", 0.3, None), (2, 2888, False, None, 0.0, None),
    (3, 4128, True, "channel", 0.0, "e2m1"), (2, 8224, True, "token", 0.1, "e4m3"), (2, 16384, True, "channel", 0.2, "e4m3"),
    (700, 288, True, "token", 0.1, None), (1300, 64, True, "channel", 0.0, "e4m3"), (333, 1056, False, "token", 0.0, None),
    (2, 16376, False, "channel", 0.0, None)]


@pytest.mark.parametrize("R,C,post,gate,p,fmt", CASES)
def test_join_and_its_gradients(R, C, post, gate, p, fmt):
    ra, rb, eps = 0.9, -0.5, 1e-5
    t, d, n, g64, mask = _case(R, C, post, gate, p, fmt, R * C)
    form = {k: d[k] for k in ("gamma_post", "gamma", "gate", "rng")} | {"residual_scale": ra, "branch_scale": rb, "p": p}
    h, y, codes, scales, r1, r2 = pgg.block_join(d["x"], d["residual"], eps=eps, fmt=fmt, **form)
    s, ry, q1, q2 = ol.join(n["x"], n["residual"], n["gamma_post"], n["gamma"], g64, ra, rb, p, mask, eps)
    mag = np.abs(s - ra * n["residual"]) + np.abs(ra * n["residual"])
    _near(h, s, mag, "h")
    ymag = (mag + np.abs(s)) * (q2[:, None] * np.abs(n["gamma"]))
    _near(y, ry, ymag, "y")
    # mean(s^2) takes each s's error: twice the ratio of the rows' magnitudes
    _near(r2, q2, q2 * (1 + np.sqrt(np.mean(mag * mag, 1)) * q2), "rstd")
    if post:
        _near(r1, q1, q1, "rstd_post")
    else:
        assert r1 is None
    if fmt:
        _check_codes(codes, scales, ry, fmt)
    rng = np.random.default_rng(3)
    dy, dh = _bf(rng, R, C), _bf(rng, R, C)
    run = lambda **kw: pgg.block_join_bwd(dy.to(DEV), dh.to(DEV), d["x"], h, r1, r2, **form, **kw)  # noqa: E731
    names = ("dx", "dresidual", "dgamma_post", "dgamma", "dgate")
    got = dict(zip(names, run()))
    ref = ol.join_bwd(_np(dy), _np(dh), n["x"], _np(h), _np(r1) if post else q1, _np(r2), n["gamma_post"], n["gamma"], g64,
                      ra, rb, p, mask)
    for name in names:
        if name in ref:
            _near(got[name], ref[name], ref["mag"][name], name)
        else:
            assert got[name] is None
    ws = torch.full((pgg.block_join_bwd_workspace_size(R, C) + 64,), 255, dtype=torch.uint8, device=DEV)
    again = dict(zip(names, run(ws=ws)))
    for name in ref["mag"]:
        assert torch.equal(got[name], again[name]), name


@pytest.mark.parametrize("R,C,post,gate,p,fmt", [
    (90, 8200, True, "channel", 0.1, None), (301, 8200, False, "token", 0.0, None), (170, 16384, True, "token", 0.0, None),
    (307, 2888, True, "token", 0.0, None), (601, 520, True, "channel", 0.0, None)])
def test_join_many_rows_a_block(R, C, post, gate, p, fmt):
    # each block, or pair of them (C > 8192), has some rows in turn, the last without a fellow in some
    test_join_and_its_gradients(R, C, post, gate, p, fmt)


def test_join_plain_is_the_norm():
    # no norm of x, no gate, no dropout: the residual's addition and the norm that the framework has
    rng = np.random.default_rng(1)
    x, r, g = (_bf(rng, *s).to(DEV) for s in ((50, 512), (50, 512), (512,)))
    h, y, codes, scales, _, rstd = pgg.block_join(x, r, gamma=g, fmt="e4m3")
    h2, y2, codes2, scales2, rstd2 = pgg.add_rmsnorm(x, r, g, fmt="e4m3")
    assert torch.equal(h, h2) and torch.equal(y, y2) and torch.equal(codes, codes2) and torch.equal(scales, scales2)
    dy, dh = _bf(rng, 50, 512).to(DEV), _bf(rng, 50, 512).to(DEV)
    dx, dr, _, dg, _ = pgg.block_join_bwd(dy, dh, x, h, None, rstd, gamma=g)
    dx2, dg2 = pgg.add_rmsnorm_bwd(dy, dh, h2, g, rstd2)
    util.assert_close(dx, util.f64(dx2), "dx", rel=2 ** -7, abs_rms=1e-5)
    assert torch.equal(dx, dr) and torch.allclose(dg, dg2, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("p", [0.0, 0.4])
def test_join_without_its_parts(p):
    """Partial outputs and operands: no residual, no next norm, no saved statistics."""
    t, d, n, g64, mask = _case(9, 264, True, "token", p, None, 5)
    form = dict(gate=d["gate"], p=p, rng=d["rng"], branch_scale=2.0)
    h, y, codes, scales, r1, r2 = pgg.block_join(d["x"], None, gamma_post=d["gamma_post"], save_rstd=False, **form)
    s, _, q1, _ = ol.join(n["x"], None, n["gamma_post"], None, g64, 1.0, 2.0, p, mask, 1e-6)
    _near(h, s, np.abs(s), "h")
    assert y is None and codes is None and scales is None and r1 is None and r2 is None
    r1 = torch.from_numpy(q1).float().to(DEV)
    dh = _bf(np.random.default_rng(1), 9, 264)
    dx, dr, dgp, dg, dgate = pgg.block_join_bwd(None, dh.to(DEV), d["x"], None, r1, None, gamma_post=d["gamma_post"],
                                                save_dresidual=False, **form)
    ref = ol.join_bwd(None, util.f64(dh), n["x"], None, _np(r1), None, n["gamma_post"], None, g64, 1.0, 2.0, p, mask)
    assert dr is None and dg is None
    for name, got in (("dx", dx), ("dgamma_post", dgp), ("dgate", dgate)):
        _near(got, ref[name], ref["mag"][name], name)
    # the norm's branch alone: no dh
    h, y, _, _, _, r2 = pgg.block_join(d["x"], d["residual"], gamma=d["gamma"])
    dx, dr, *_ = pgg.block_join_bwd(dh.to(DEV), None, d["x"], h, None, r2, gamma=d["gamma"])
    ref = ol.join_bwd(util.f64(dh), None, n["x"], _np(h), None, _np(r2), None, n["gamma"], None, 1.0, 1.0, 0.0,
                      np.ones((9, 264), bool))
    _near(dx, ref["dx"], ref["mag"]["dx"], "dx")
    _near(dr, ref["dresidual"], ref["mag"]["dresidual"], "dresidual")


def test_join_dropped_places_hold_nothing():
    # infinities and NaN where the mask drops; rows that it leaves empty
    R, C, p = 64, 32, 0.9
    t, d, n, _, mask = _case(R, C, False, None, p, None, 11)
    x = d["x"].clone()
    bad = torch.from_numpy(~mask).to(DEV)
    x[bad] = torch.tensor(float("nan"), dtype=BF, device=DEV)
    x[bad & (torch.arange(C, device=DEV) % 2 == 0)] = float("-inf")
    h, y, *_, r2 = pgg.block_join(x, d["residual"], gamma=d["gamma"], p=p, rng=d["rng"])
    ref, yref, *_ = pgg.block_join(d["x"], d["residual"], gamma=d["gamma"], p=p, rng=d["rng"])
    assert torch.equal(h, ref) and torch.equal(y, yref)
    empty = ~mask.any(axis=1)
    assert empty.any()
    assert torch.equal(h[torch.from_numpy(empty).to(DEV)], d["residual"][torch.from_numpy(empty).to(DEV)])
    dy = torch.ones_like(x)
    dx, *_ = pgg.block_join_bwd(dy, dy, x, h, None, r2, gamma=d["gamma"], p=p, rng=d["rng"])
    assert torch.isfinite(dx).all() and (dx[bad] == 0).all()


def test_join_dropped_places_of_a_row_without_a_norm():
    # a NaN or an infinity in a row that is normed: its kept elements have no value, its dropped ones are 0
    R, C, p = 24, 264, 0.5
    t, d, n, _, mask = _case(R, C, True, "token", p, None, 12)
    x = d["x"].clone()
    x[3, 7], x[4, 9], x[5, 250] = float("nan"), float("inf"), float("-inf")
    form = {k: d[k] for k in ("gamma_post", "gate", "rng")} | {"p": p}
    h, *_ = pgg.block_join(x, d["residual"], **form)
    ref, *_ = pgg.block_join(d["x"], d["residual"], **form)
    keep = torch.from_numpy(mask).to(DEV)
    assert torch.equal(h[~keep], d["residual"][~keep])
    assert torch.isnan(h[3][keep[3]]).all()
    rest = torch.ones(R, dtype=torch.bool, device=DEV)
    rest[3:6] = False
    assert torch.equal(h[rest], ref[rest])
    # a row that the mask empties is the residual's, and so is its norm
    p, x, res = 0.9, d["x"][:, :8].contiguous(), d["residual"][:, :8].contiguous()
    keep = torch.from_numpy(ol.keep(R, 8, p, t["rng"].tolist())).to(DEV)
    empty = ~keep.any(dim=1)
    assert empty.any()
    x[empty, 5] = float("nan")
    one = torch.ones(8, dtype=BF, device=DEV)
    h, y, *_ = pgg.block_join(x, res, gamma_post=one, gamma=one, p=p, rng=d["rng"])
    assert torch.equal(h[empty], res[empty])
    assert torch.equal(y[empty], pgg.block_join(torch.zeros_like(x), res, gamma=one)[1][empty])


def test_join_rows_of_zeros_and_special_values():
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    g = torch.ones(64, dtype=BF, device=DEV)
    h, y, codes, scales, r1, r2 = pgg.block_join(x, torch.zeros_like(x), gamma_post=g, gamma=g, fmt="e4m3")
    assert (h[[0, 3]] == 0).all() and (y[[0, 3]] == 0).all() and (codes[[0, 3]] == 0).all()
    assert r1[0].item() == pytest.approx(1e3, rel=1e-6) and torch.isnan(h[2]).all() and (scales[2] == 255).all()
    assert torch.isnan(h[1, 3]) and (h[1, :3] == 0).all()   # inf * 0, and 0 * 0


def test_join_in_place():
    _in_place(300, 520)


def test_join_in_place_on_clusters():
    _in_place(130, 8264)


def _in_place(R, C):
    t, d, n, _, mask = _case(R, C, True, "channel", 0.2, None, 21)
    form = {k: d[k] for k in ("gamma_post", "gamma", "gate", "rng")} | {"p": 0.2}
    h, y, _, _, r1, r2 = pgg.block_join(d["x"], d["residual"], **form)
    for name in ("x", "residual"):
        a = {k: d[k].clone() for k in ("x", "residual")}
        h2, y2, *_ = pgg.block_join(a["x"], a["residual"], h=a[name], **form)
        assert torch.equal(h, h2) and torch.equal(y, y2)
    dy, dh = (_bf(np.random.default_rng(s), R, C).to(DEV) for s in (1, 2))
    ref = pgg.block_join_bwd(dy, dh, d["x"], h, r1, r2, **form)
    for first, second in (("dy", "dh"), ("x", "h"), ("dh", "dy"), ("h", "x")):
        a = {"dy": dy.clone(), "dh": dh.clone(), "x": d["x"].clone(), "h": h.clone()}
        got = pgg.block_join_bwd(a["dy"], a["dh"], a["x"], a["h"], r1, r2, dx=a[first], dresidual=a[second], **form)
        for u, v in zip(ref, got):
            assert torch.equal(u, v)


def test_join_in_a_graph_follows_the_generator_state():
    t, d, n, _, _ = _case(40, 256, True, None, 0.3, None, 31)
    form = {k: d[k] for k in ("gamma_post", "gamma", "rng")} | {"p": 0.3}
    pgg.block_join(d["x"], d["residual"], **form)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h, y, _, _, r1, r2 = pgg.block_join(d["x"], d["residual"], **form)
        grads = pgg.block_join_bwd(y, h, d["x"], h, r1, r2, **form)
    seen = []
    for _ in range(3):
        d["rng"][1] += 1
        g.replay()
        eager = pgg.block_join(d["x"], d["residual"], **form)
        assert torch.equal(h, eager[0]) and torch.equal(y, eager[1])
        for a, b in zip(grads, pgg.block_join_bwd(y, h, d["x"], h, r1, r2, **form)):
            assert a is b or torch.equal(a, b)
        seen.append(h.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_join_on_another_stream_and_empty():
    t, d, *_ = _case(600, 1056, True, "token", 0.1, None, 41)
    form = {k: d[k] for k in ("gamma_post", "gamma", "gate", "rng")} | {"p": 0.1}
    ref = pgg.block_join(d["x"], d["residual"], **form)
    rb = pgg.block_join_bwd(ref[1], ref[0], d["x"], ref[0], ref[4], ref[5], **form)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pgg.block_join(d["x"], d["residual"], stream=s, **form)
    gb = pgg.block_join_bwd(got[1], got[0], d["x"], got[0], got[4], got[5], stream=s, **form)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref + rb, got + gb) if a is not None)
    e = torch.zeros(0, 64, dtype=BF, device=DEV)
    gm = torch.ones(64, dtype=BF, device=DEV)
    z = torch.zeros(0, device=DEV)
    h, y, *_ = pgg.block_join(e, e, gamma_post=gm, gamma=gm)
    assert h.shape == (0, 64)
    dx, dr, d1, d2, dg = pgg.block_join_bwd(e, e, e, h, z, z, gamma_post=gm, gamma=gm, gate=gm)
    assert (d1 == 0).all() and (d2 == 0).all() and (dg == 0).all() and dg.shape == (64,)


def test_join_on_three_streams_at_once():
    # rows of a thread's one, of two pieces, and of a cluster; with a product between them
    work = []
    for seed, (R, C) in enumerate(((700, 520), (500, 4096), (400, 8200))):
        rng = np.random.default_rng(seed)
        t = {k: _bf(rng, R, C).to(DEV) for k in ("x", "residual", "dy", "dh")}
        w = _bf(rng, 64, C, scale=C ** -0.5).to(DEV)
        form = {"gamma_post": _bf(rng, C).to(DEV), "gamma": _bf(rng, C).to(DEV), "gate": _bf(rng, C).to(DEV), "p": 0.1,
                "rng": torch.tensor([seed, 5], device=DEV)}
        work.append((t, w, form))

    def run(t, w, form):
        h, y, _, _, r1, r2 = pgg.block_join(t["x"], t["residual"], **form)
        z, _ = pgg.grouped_linear(y[:24], w)
        return (h, y, z, *pgg.block_join_bwd(t["dy"], t["dh"], t["x"], h, r1, r2, **form))

    ref = [run(*a) for a in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = []
    for _ in range(6):
        for st, a in zip(streams, work):
            with torch.cuda.stream(st):
                got.append(run(*a))
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert all(torch.equal(u, v) for u, v in zip(out, ref[i % 3]))


def test_join_mask_past_32_bits_of_elements():
    # rows whose element index passes 2^32 (the counter's words carry on): one kept share, other bits
    R, C = 262200, 16384
    x = torch.ones(1, C, dtype=BF, device=DEV).expand(R, C)
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * R * C * 2:
        pytest.skip("needs 26 GB of device memory")
    x = x.contiguous()
    rng = torch.tensor([5, 6], device=DEV)
    h, *_ = pgg.block_join(x, None, p=0.5, rng=rng)
    for row in (0, 262143, 262144, R - 1):
        words = [w for i in range(row * C // 4, row * C // 4 + 16)
                 for w in ol.philox4x32((i & 0xFFFFFFFF, i >> 32, 6, 0), (5, 0))]
        np.testing.assert_array_equal(h[row, :64].float().cpu().numpy(), np.where(np.array(words) >= 2 ** 31, 2.0, 0.0))
