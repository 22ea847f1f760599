"""GPU parity of the operators around the grouped GEMMs -- norm, router, few-token layer -- with the
fp64 oracle.

Tolerances, from the arithmetic: a bf16 output is one rounding (2^-9 relative) of an fp32 value
whose own error is far smaller, so 2^-8 |ref| plus 2^-16 of the magnitudes that were summed; fp32
outputs 2^-18 of the same.  Choices of experts are equal.  MX codes come from an fp32 value that may
sit on the other side of a rounding boundary than the fp64 one: at most one code in a thousand may
differ, by one step of the grid.  After an MX rounding in the middle (the activation of the
few-token layer) one activation of each output may be such a step off: 1/8 of its term in e4m3, 1/2
in e2m1."""

import time

import numpy as np
import pytest
import torch

from oracle import block as ob
from oracle import grouped_gemm as og
from oracle import moe_glue as mg
from oracle import mx as omx
from precision_grouped_gemm_gb300 import _binding
import util

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _close(got, ref, mag, rel, what):
    """|got - ref| <= rel |ref| + 2^-16 (bf16) or 2^-18 (fp32) mag, and the same NaNs."""
    g = got.detach().cpu().double().numpy()
    tiny = 2.0 ** (-16 if got.dtype == BF else -18)
    bound = rel * np.abs(ref) + tiny * mag + 1e-30
    assert np.array_equal(np.isnan(g), np.isnan(ref)), f"{what}: other NaNs"
    err = np.where(np.isnan(ref), 0.0, np.abs(g - ref))
    bad = ~(err <= np.where(np.isnan(ref), 1.0, bound))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(err / bound):.3g} of the bound"


BF16_REL, F32_REL = 2.0 ** -8, 2.0 ** -18


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(BF)


# ---------------------------------------------------------------- norm

def _check_codes(codes, scales, y, fmt):
    """Codes and scales of fp64 rows y, up to boundary cases."""
    R, C = y.shape
    rs, rc = omx.quantize_blocks(fmt, y.reshape(R, C // 32, 32))
    gs = scales.cpu().numpy()
    gc = codes.cpu().numpy()
    gc = (omx.unpack_e2m1(gc) if fmt == "e2m1" else gc).reshape(R, C // 32, 32)
    assert np.mean(gs != rs) <= 1e-3
    same = gs == rs
    a, b = gc[same].astype(int), rc[same].astype(int)
    assert np.mean(a != b) <= 1e-3 and np.abs(a - b).max(initial=0) <= 1


NORMS = [(1, 32, True, "e4m3"), (3, 96, False, "e2m1"), (5, 1056, True, "e4m3"), (2, 16384, True, "e2m1"),
         (7, 4096, True, "e4m3"), (700, 288, True, "e4m3"), (2, 8, True, None), (9, 2888, False, None),
         (1200, 2048, True, "e2m1"), (3, 8224, True, "e4m3")]


@pytest.mark.parametrize("R,C,residual,fmt", NORMS)
def test_add_rmsnorm(R, C, residual, fmt):
    rng = np.random.default_rng(R * C)
    x, r, g = _bf(rng, R, C), _bf(rng, R, C, scale=3.0) if residual else None, _bf(rng, C)
    h, y, codes, scales, rstd = pgg.add_rmsnorm(x.to(DEV), r.to(DEV) if residual else None, g.to(DEV), 1e-5, fmt=fmt)
    s, ry, rr = ob.add_rmsnorm(util.f64(x), util.f64(r) if residual else None, util.f64(g), 1e-5)
    _close(h, s, np.abs(s), BF16_REL, "h")
    _close(y, ry, np.abs(ry), BF16_REL, "y")
    _close(rstd, rr, rr, F32_REL, "rstd")
    if fmt:
        _check_codes(codes, scales, ry, fmt)
    else:
        assert codes is None and scales is None


@pytest.mark.parametrize("R,C,residual,_", NORMS)
def test_add_rmsnorm_bwd(R, C, residual, _):
    rng = np.random.default_rng(R + C)
    h, g, dy = _bf(rng, R, C, scale=2.0), _bf(rng, C), _bf(rng, R, C)
    dh = _bf(rng, R, C) if residual else None
    rstd = torch.from_numpy((1 / np.sqrt(np.mean(util.f64(h) ** 2, axis=1) + 1e-5)).astype(np.float32))
    dx, dg = pgg.add_rmsnorm_bwd(dy.to(DEV), dh.to(DEV) if residual else None, h.to(DEV), g.to(DEV), rstd.to(DEV))
    a = [util.f64(dy), util.f64(dh) if residual else None, util.f64(h), util.f64(g), rstd.double().numpy()]
    rdx, rdg = ob.add_rmsnorm_bwd(*a)
    u, xh = np.abs(a[0] * a[3]), np.abs(a[2] * a[4][:, None])
    mag = a[4][:, None] * (u + xh * np.mean(u * xh, axis=1, keepdims=True)) + (np.abs(a[1]) if residual else 0)
    _close(dx, rdx, mag, BF16_REL, "dx")
    _close(dg, rdg, np.sum(np.abs(a[0]) * xh, axis=0), F32_REL, "dgamma")
    dx2, dg2 = pgg.add_rmsnorm_bwd(dy.to(DEV), dh.to(DEV) if residual else None, h.to(DEV), g.to(DEV), rstd.to(DEV))
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)  # a fixed order


def test_add_rmsnorm_gradient_against_differences():
    # the GPU forward in fp64-sized steps is not possible; its gradient is compared with central
    # differences of the oracle's forward at the GPU's own h and rstd
    rng = np.random.default_rng(5)
    R, C = 6, 160
    x, g, dy = _bf(rng, R, C), _bf(rng, C), _bf(rng, R, C)
    h, _, _, _, rstd = pgg.add_rmsnorm(x.to(DEV), None, g.to(DEV), 1e-3)
    dx, dg = pgg.add_rmsnorm_bwd(dy.to(DEV), None, h, g.to(DEV), rstd)
    f = lambda z, q: np.sum(ob.add_rmsnorm(z, None, q, 1e-3)[1] * util.f64(dy))  # noqa: E731
    v, q, e = rng.standard_normal((R, C)), rng.standard_normal(C), 1e-5
    x64, g64 = util.f64(x), util.f64(g)
    num = (f(x64 + e * v, g64) - f(x64 - e * v, g64)) / (2 * e)
    # the bf16 rounding of R C gradients, added up at random signs: 2^-9 of the norm of dx v
    bound = 4 * 2.0 ** -9 * np.linalg.norm(util.f64(dx) * v)
    assert abs(np.sum(util.f64(dx) * v) - num) <= bound
    num = (f(x64, g64 + e * q) - f(x64, g64 - e * q)) / (2 * e)
    assert np.sum(dg.double().cpu().numpy() * q) == pytest.approx(num, rel=1e-5)


def test_add_rmsnorm_edge_rows():
    # zero rows (h, y, codes 0; scale code 0), a NaN and an infinity that stay in their rows, huge values
    C = 64
    x = torch.zeros(5, C, dtype=BF)
    x[1] = 1.0
    x[1, 40] = float("nan")
    x[2] = 1.0
    x[2, 3] = float("inf")
    x[3] = 1e18
    x[4] = 2.0
    h, y, codes, scales, rstd = pgg.add_rmsnorm(x.to(DEV), None, torch.ones(C, dtype=BF, device=DEV), 1e-6, fmt="e4m3")
    assert not y[0].any() and not codes[0].any() and not scales[0].any()
    assert torch.isnan(y[1]).all() and (scales[1] == 255).all() and not codes[1].any()
    assert torch.isnan(y[2, 3]) and not y[2, :3].any()       # inf / inf; finite / inf
    assert scales[2, 0] == 255 and scales[2, 1] == 0
    assert torch.allclose(y[3].float(), torch.ones(C, device=DEV), rtol=2 ** -7)
    assert torch.equal(y[4].float(), torch.ones(C, device=DEV)) and torch.isfinite(rstd[3:]).all()


def test_add_rmsnorm_in_place_empty_and_partial_outputs():
    rng = np.random.default_rng(8)
    x, r, g = _bf(rng, 33, 256).to(DEV), _bf(rng, 33, 256).to(DEV), _bf(rng, 256).to(DEV)
    h, y, c, s, _ = pgg.add_rmsnorm(x, r, g, fmt="e4m3")
    xi, ri = x.clone(), r.clone()
    assert pgg.add_rmsnorm(xi, r, g, h=xi)[0] is xi and torch.equal(xi, h)       # the sum over x
    h2, y2, c2, s2, q2 = pgg.add_rmsnorm(x, ri, g, h=ri, fmt="e4m3", save_y=False, save_rstd=False)
    assert torch.equal(ri, h) and y2 is None and q2 is None and torch.equal(c, c2) and torch.equal(s, s2)
    e = torch.empty(0, 256, dtype=BF, device=DEV)
    assert pgg.add_rmsnorm(e, e, g, fmt="e4m3")[1].shape == (0, 256)
    dx, dg = pgg.add_rmsnorm_bwd(e, None, e, g, torch.empty(0, device=DEV))
    assert dx.shape == (0, 256) and not dg.any()
    dy, rstd = _bf(rng, 33, 256).to(DEV), torch.ones(33, device=DEV)
    ref, _ = pgg.add_rmsnorm_bwd(dy, x, h, g, rstd)
    xi = x.clone()
    assert torch.equal(pgg.add_rmsnorm_bwd(dy, xi, h, g, rstd, dx=xi)[0], ref)   # the gradient over dh


def test_norm_codes_feed_the_grouped_gemm():
    # the norm's MX output is the operand of the block-scaled forward GEMM
    rng = np.random.default_rng(9)
    M, K, N = 70, 256, 128
    x, g, W = _bf(rng, M, K), _bf(rng, K), _bf(rng, 2 * N, K, scale=0.1)
    lens = torch.tensor([40, 30], dtype=torch.int32, device=DEV)
    _, _, c, s, _ = pgg.add_rmsnorm(x.to(DEV), None, g.to(DEV), fmt="e4m3")
    wc, ws = pgg.mx_quantize_rowwise_blocked(W.to(DEV), "e4m3")
    out = pgg.mx_grouped_gemm(pgg.MODE_FWD, "e4m3", c, s, wc, ws, lens, M, N, K)
    wr, wsr = omx.mx_quantize_rowwise(util.bits(W), "e4m3")
    ref = omx.mx_grouped_gemm_fwd("e4m3", c.cpu().numpy(), s.cpu().numpy(), wr, wsr, [40, 30], 2)
    util.assert_close(out, ref, "grouped GEMM on the norm's codes")


# ---------------------------------------------------------------- router

ROUTES = [  # T, E, k, dtype, score, renormalize, bias, masked
    (1, 1, 1, "f32", "softmax", True, False, 0), (5, 8, 8, "bf16", "softmax", False, False, 2),
    (33, 31, 3, "f32", "sigmoid", True, True, 4), (130, 33, 2, "bf16", "sigmoid", False, True, 0),
    (64, 64, 6, "f32", "softmax", True, True, 5), (257, 100, 4, "bf16", "softmax", True, False, 0),
    (90, 256, 8, "f32", "sigmoid", True, True, 32), (40, 500, 10, "f32", "softmax", False, True, 3),
    (17, 1024, 32, "bf16", "softmax", False, False, 100), (21, 1000, 16, "f32", "sigmoid", False, False, 0)]


def _logits(T, E, dtype, bias, masked, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32) * 2)
    if masked:
        x[:, torch.from_numpy(rng.choice(E, masked, replace=False))] = -float("inf")
    if dtype == "bf16":
        x = x.to(BF)
    return x, torch.from_numpy(rng.standard_normal(E).astype(np.float32)) if bias else None


def _np(x):
    return x.float().numpy()


@pytest.mark.parametrize("T,E,k,dtype,score,renormalize,bias,masked", ROUTES)
def test_moe_route(T, E, k, dtype, score, renormalize, bias, masked):
    x, b = _logits(T, E, dtype, bias, masked, T + E)
    ids, w = pgg.moe_route(x.to(DEV), k, None if b is None else b.to(DEV), score, renormalize, 2.5)
    rid, rw = ob.moe_route(_np(x), None if b is None else b.numpy(), k, score, renormalize, 2.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    _close(w, rw, np.abs(rw), F32_REL, "w")
    rng = np.random.default_rng(T)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    d = pgg.moe_route_bwd(x.to(DEV), ids, dw.to(DEV), None if b is None else b.to(DEV), score, renormalize, 2.5)
    ref = ob.moe_route_bwd(_np(x), None if b is None else b.numpy(), rid, dw.double().numpy(), score, renormalize, 2.5)
    assert d.dtype == x.dtype
    mag = 2.5 * np.abs(dw.double().numpy()).sum(1, keepdims=True) * np.ones_like(ref)
    _close(d, ref, mag, BF16_REL if dtype == "bf16" else F32_REL, "dlogits")


def test_moe_route_masked_rows_nan_inf_and_ties():
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[-inf] * 6,                       # masked whole: ids 0.., weights 0
                      [-inf, -inf, 1.0, -inf, -inf, 0.0],  # fewer than k left
                      [0.0, nan, 2.0, 1.0, -inf, 0.0],  # NaN: ranked last, weights NaN
                      [-0.0, 0.0, -0.0, 0.0, -1.0, 0.0],  # -0 and +0 tie
                      [torch.finfo(torch.float32).min] * 6,  # a mask by the type's lowest value
                      [100.0, -100.0, 100.0, 100.0, -100.0, 99.0]])
    for dt in (torch.float32, BF):
        for score in ("softmax", "sigmoid"):
            for renorm in (True, False):
                z = x.to(dt)
                ids, w = pgg.moe_route(z.to(DEV), 3, None, score, renorm)
                rid, rw = ob.moe_route(_np(z), None, 3, score, renorm, 1.0)
                np.testing.assert_array_equal(ids.cpu().numpy(), rid)
                _close(w, rw, np.abs(rw), F32_REL, f"w {score} {renorm}")
                dw = torch.ones(6, 3)
                d = pgg.moe_route_bwd(z.to(DEV), ids, dw.to(DEV), None, score, renorm)
                ref = ob.moe_route_bwd(_np(z), None, rid, dw.double().numpy(), score, renorm, 1.0)
                _close(d, ref, 3.0 * np.ones_like(ref), BF16_REL if dt == BF else F32_REL, f"d {score} {renorm}")
    ids, w = pgg.moe_route(torch.tensor([[1.0, inf, 0.0]], device=DEV), 2)
    assert ids.tolist() == [[1, 0]] and torch.isnan(w[0, 0]) and w[0, 1] == 0    # inf - inf, as the formula has it
    bias = torch.tensor([0.0, -inf, 0.0, 0.0], device=DEV)                     # the bias masks expert 1
    ids, w = pgg.moe_route(torch.tensor([[0.0, 9.0, 1.0, 1.0]], device=DEV), 4, bias, "sigmoid", True)
    assert ids.tolist() == [[2, 3, 0, 1]] and w[0, 3] == 0
    assert pgg.moe_route(torch.empty(0, 8, device=DEV), 2)[0].shape == (0, 2)


@pytest.mark.parametrize("T,E,k", [(1025, 8, 8), (1026, 8, 1), (1027, 16, 3), (1100, 72, 7), (1031, 256, 8),
                                   (1028, 512, 6), (1029, 1024, 8)])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("dtype,bias", [("bf16", False), ("bf16", True), ("f32", False), ("f32", True)])
def test_moe_route_many_tokens(T, E, k, score, renormalize, dtype, bias):
    rng = np.random.default_rng(T + E)
    # few different values, so that most choices are ties; masked places, a NaN row, a row masked whole
    x = torch.from_numpy(rng.integers(-4, 5, (64, E)).astype(np.float32) / 2)
    x[torch.from_numpy(rng.random((64, E)) < 0.2)] = -float("inf")
    x[11, E // 3] = float("nan")
    x[20] = -float("inf")
    rows = rng.integers(0, 64, T)
    rows[-3:] = (11, 20, 5)
    x = x.to(BF if dtype == "bf16" else torch.float32)
    b = torch.from_numpy(rng.integers(-4, 5, E).astype(np.float32) / 2) if bias else None
    ids, w = pgg.moe_route(x[rows].to(DEV), k, None if b is None else b.to(DEV), score, renormalize, 2.5)
    rid, rw = ob.moe_route(_np(x), None if b is None else b.numpy(), k, score, renormalize, 2.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid[rows])
    _close(w, rw[rows], np.abs(rw[rows]), F32_REL, "w")


def test_moe_route_bf16_every_value():
    # every bf16 value but the NaNs, in rows of 256 in random order: signs, zeros, subnormals, infinities
    v = np.arange(65536, dtype=np.uint16)
    v = np.random.default_rng(3).permutation(v[(v & 0x7FFF) <= 0x7F80])
    v = v[:len(v) // 256 * 256].reshape(-1, 256)
    x = torch.from_numpy(v.astype(np.int32) << 16).view(torch.float32).to(BF)
    for E, times in ((256, 1), (256, 5), (255, 5)):  # few tokens and many; in whole chunks, and not
        y = x[:, :E].contiguous()
        ids, w = pgg.moe_route(y.repeat(times, 1).to(DEV), 8, None, "sigmoid", True)
        rid, rw = ob.moe_route(_np(y), None, 8, "sigmoid", True, 1.0)
        np.testing.assert_array_equal(ids.cpu().numpy(), np.tile(rid, (times, 1)))
        _close(w, np.tile(rw, (times, 1)), np.abs(np.tile(rw, (times, 1))), F32_REL, "w")


@pytest.mark.parametrize("T", [3, 1027])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_moe_route_chosen_far_below(T, dtype):
    # the bias chooses experts whose scores are below fp32's range next to the largest logit's:
    # the renormalised weights do not depend on that
    x = torch.full((T, 8), 3.0)
    x[:, 2], x[:, 5], x[:, 7] = -200.0, -201.0, -199.0
    b = torch.full((8,), -1000.0)
    b[2], b[5], b[7] = 0.0, 1.0, 0.5
    x = x.to(BF if dtype == "bf16" else torch.float32)
    ids, w = pgg.moe_route(x.to(DEV), 3, b.to(DEV), "softmax", True)
    rid, rw = ob.moe_route(_np(x), b.numpy(), 3, "softmax", True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    _close(w, rw, np.abs(rw), F32_REL, "w")
    dw = torch.tensor([[1.0, -2.0, 0.5]]).repeat(T, 1)
    d = pgg.moe_route_bwd(x.to(DEV), ids, dw.to(DEV), b.to(DEV), "softmax", True)
    ref = ob.moe_route_bwd(_np(x), b.numpy(), rid, dw.double().numpy(), "softmax", True, 1.0)
    _close(d, ref, 3.5 * np.ones_like(ref), BF16_REL if dtype == "bf16" else F32_REL, "dlogits")


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", False)])
def test_moe_route_bwd_masked_choice_has_no_part(score, renormalize):
    # two experts left of eight: the third choice is masked, and its dw (here not a number) is not used
    x = torch.full((5, 8), -float("inf"))
    x[:, 3], x[:, 6] = 0.5, -0.25
    ids, _ = pgg.moe_route(x.to(DEV), 3, None, score, renormalize)
    dw = torch.tensor([[1.0, 2.0, 0.0]]).repeat(5, 1)
    ref = ob.moe_route_bwd(_np(x), None, ids.cpu().numpy(), dw.double().numpy(), score, renormalize, 1.0)
    dw[:, 2] = float("nan")
    d = pgg.moe_route_bwd(x.to(DEV), ids, dw.to(DEV), None, score, renormalize)
    _close(d, ref, 3.0 * np.ones_like(ref), F32_REL, "dlogits")


def test_moe_route_bwd_ids_of_other_kinds():
    # an id out of range has no part; an expert named twice gets both terms
    x = torch.tensor([[0.5, -1.0, 2.0, 0.0]], device=DEV)
    ids = torch.tensor([[2, 7, -1, 2]], dtype=torch.int32, device=DEV)
    dw = torch.tensor([[1.0, 5.0, 5.0, 2.0]], device=DEV)
    d = pgg.moe_route_bwd(x, ids, dw, score="sigmoid", renormalize=False)
    s = 1 / (1 + np.exp(-2.0))
    np.testing.assert_allclose(d.cpu().numpy(), [[0, 0, 3 * s * (1 - s), 0]], rtol=1e-5)


# ---------------------------------------------------------------- few-token layer

def _layer(T, k, E, H, I, fmt, seed, distinct=True, skew=0.0):
    """Inputs on the CPU, the call's arguments on the GPU, and the oracle's operands."""
    rng = np.random.default_rng(seed)
    p = np.arange(1, E + 1, dtype=np.float64) ** -skew
    p /= p.sum()
    if distinct:
        ids = np.argsort(-(np.log(p) - np.log(-np.log(rng.random((T, E))))), axis=1)[:, :k].astype(np.int32)
    else:
        ids = rng.choice(E, size=(T, k), p=p).astype(np.int32)
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32))
    x = _bf(rng, T, H)
    W1, W2 = _bf(rng, E * 2 * I, H, scale=H ** -0.5), _bf(rng, E * H, I, scale=I ** -0.5)
    gid = torch.from_numpy(ids).to(DEV)
    if fmt is None:
        dev = (x.to(DEV), gid, w.to(DEV), W1.view(E, 2 * I, H).to(DEV), W2.view(E, H, I).to(DEV))
        ref = (util.f64(x), util.f64(W1).reshape(E, 2 * I, H), util.f64(W2).reshape(E, H, I))
    else:
        q = lambda t: omx.mx_dequantize(*omx.mx_quantize_rowwise(util.bits(t), fmt), fmt)  # noqa: E731
        dev = (fmt, *pgg.mx_quantize_rowwise(x.to(DEV), fmt), gid, w.to(DEV),
               *pgg.mx_quantize_rowwise_blocked(W1.to(DEV), fmt), *pgg.mx_quantize_rowwise_blocked(W2.to(DEV), fmt))
        ref = (q(x), q(W1).reshape(E, 2 * I, H), q(W2).reshape(E, H, I))
    return ids, w, dev, ref


def _call(fmt, dev, **kw):
    return (pgg.moe_decode if fmt is None else pgg.mx_moe_decode)(*dev, **kw)


def _check_layer(out, ids, w, ref, fmt, limit=None):
    x, W1, W2 = ref
    r, top, mag = ob.moe_decode(x, ids, None if w is None else w.double().numpy(), W1, W2, limit, fmt)
    g = out.detach().cpu().double().numpy()
    # fp32 accumulation and the two-part bf16 activation: 2^-14 of the summed magnitudes
    bound = 2.0 ** -8 * np.abs(r) + 2.0 ** -14 * mag + {None: 0.0, "e4m3": 0.125, "e2m1": 0.5}[fmt] * top
    err = np.abs(g - r)
    assert (err <= bound).all(), f"worst {np.max(err / bound):.3g} of the bound"
    return r


BF16_LAYERS = [(1, 2, 8, 256, 256), (3, 4, 7, 72, 200), (33, 3, 5, 264, 136), (64, 6, 16, 512, 384), (128, 4, 8, 256, 128),
               (17, 32, 40, 64, 72), (2, 1, 1, 8, 8), (128, 2, 1024, 64, 64), (5, 3, 300, 1000, 1032)]
MX_LAYERS = [(1, 2, 8, 256, 256), (5, 3, 9, 384, 640), (33, 3, 5, 128, 256), (64, 6, 16, 512, 384),
             (128, 4, 8, 256, 128), (17, 32, 40, 128, 128), (90, 1, 2, 640, 128)]


@pytest.mark.parametrize("T,k,E,H,I", BF16_LAYERS)
@pytest.mark.parametrize("limit", [0.0, 0.5])
def test_moe_decode(T, k, E, H, I, limit):
    ids, w, dev, ref = _layer(T, k, E, H, I, None, T * 7 + E)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pgg.moe_decode(*dev, swiglu_limit=limit, err=err)
    assert pgg.read_error(err) == 0
    _check_layer(out, ids, w, ref, None, limit or None)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("T,k,E,H,I", MX_LAYERS)
def test_mx_moe_decode(T, k, E, H, I, fmt):
    limit = 0.0 if T % 2 else 1.0
    ids, w, dev, ref = _layer(T, k, E, H, I, fmt, T * 5 + E)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pgg.mx_moe_decode(*dev, swiglu_limit=limit, err=err)
    assert pgg.read_error(err) == 0
    _check_layer(out, ids, w, ref, fmt, limit or None)


@pytest.mark.parametrize("fmt", [None, "e4m3", "e2m1"])
@pytest.mark.parametrize("T,k,E", [(9, 4, 1000), (2, 32, 200), (12, 3, 1024)])
def test_decode_many_experts_few_tokens(T, k, E, fmt):
    ids, w, dev, ref = _layer(T, k, E, 128, 128, fmt, T + E)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(3):
        out = _call(fmt, dev, err=err)
        assert pgg.read_error(err) == 0
        _check_layer(out, ids, w, ref, fmt)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_calls_on_another_stream_than_the_current_one(fmt):
    # what a call makes for itself (outputs, workspaces and their zeros) is in the order of its stream,
    # not behind or ahead of the current stream's work
    ids, w, dev, ref = _layer(6, 3, 8, 256, 128, fmt, 5)
    x, g = _bf(np.random.default_rng(2), 40, 256).to(DEV), torch.ones(256, dtype=BF, device=DEV)
    logits = torch.randn(50, 16, device=DEV)
    here = pgg.add_rmsnorm(x, x, g), pgg.moe_route(logits, 4)
    back = pgg.add_rmsnorm_bwd(x, None, here[0][0], g, here[0][4])
    big = torch.randn(8192, 8192, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    filler = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    del filler  # the current stream's next small blocks are not zero
    for _ in range(20):
        big = big @ big * 1e-4  # the current stream is busy
    out = _call(fmt, dev, stream=side)
    there = pgg.add_rmsnorm(x, x, g, stream=side), pgg.moe_route(logits, 4, stream=side)
    bside = pgg.add_rmsnorm_bwd(x, None, there[0][0], g, there[0][4], stream=side)
    side.synchronize()
    _check_layer(out, ids, w, ref, fmt)
    for a, b in zip([*here[0], *here[1], *back], [*there[0], *there[1], *bside]):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))


@pytest.mark.parametrize("fmt", [None, "e4m3", "e2m1"])
def test_decode_skewed_and_repeated_experts(fmt):
    # most tokens on one expert, and tokens that name an expert several times: the weights add up
    ids, w, dev, ref = _layer(60, 5, 12, 256, 256, fmt, 11, distinct=False, skew=2.0)
    assert max(np.bincount(ids.reshape(-1), minlength=12)) > 64 and any(len(set(r)) < 5 for r in ids.tolist())
    _check_layer(_call(fmt, dev), ids, w, ref, fmt)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_decode_bad_ids_no_weights_and_empty(fmt):
    ids, w, dev, ref = _layer(9, 3, 6, 256, 128, fmt, 12)
    at = 1 if fmt is None else 3  # where the ids stand among the arguments
    bad = ids.copy()
    bad[2, 1], bad[4] = 6, -1
    call = list(dev)
    call[at] = torch.from_numpy(bad).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = _call(fmt, call, err=err)
    assert pgg.read_error(err) == 19
    assert not out[4].any()                      # a token without an expert
    _check_layer(out, bad, w, ref, fmt)
    call[at] = torch.full_like(call[at], -1)     # a batch without one: zeros, whatever was there
    out.fill_(7.0)
    assert not _call(fmt, call, out=out).any()
    call = list(dev)
    call[at + 1] = None                          # no weights: 1 each
    _check_layer(_call(fmt, call), ids, None, ref, fmt)
    call = list(dev)
    for i in ((0, 1, 2) if fmt is None else (1, 2, 3, 4)):
        call[i] = call[i][:0]                    # no tokens
    assert _call(fmt, call).shape == (0, 256)


def test_decode_nan_stays_with_its_token():
    ids, w, dev, ref = _layer(20, 2, 4, 256, 128, None, 13)
    good = pgg.moe_decode(*dev)
    x = dev[0].clone()
    x[7, 100] = float("nan")
    out = pgg.moe_decode(x, *dev[1:])
    assert torch.isnan(out[7]).all()
    keep = [t for t in range(20) if t != 7]
    assert torch.equal(out[keep], good[keep])


def test_decode_workspace_is_left_ready_and_results_repeat():
    # one workspace for calls of several sizes; its counters are zero again after each; the same bits
    # on every run, on another stream, and from a graph
    cases = [(fmt, _layer(T, k, E, H, I, fmt, T))
             for fmt, T, k, E, H, I in ((None, 40, 4, 16, 512, 256), ("e2m1", 3, 2, 5, 256, 384), (None, 1, 3, 9, 264, 72),
                                        ("e4m3", 64, 4, 7, 128, 128))]
    ws = pgg.moe_decode_workspace(64, 4, 512, 1024, 16)
    first = [_call(f, c[2], ws=ws) for f, c in cases]
    assert not ws[:4096].any()
    for (f, c), o in zip(cases, first):
        _check_layer(o, c[0], c[1], c[3], f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [_call(f, c[2], ws=ws) for f, c in cases]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    out = torch.zeros_like(first[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(None, cases[0][1][2], ws=ws, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0])


@pytest.mark.parametrize("fmt", [None, "e4m3", "e2m1"])
@pytest.mark.parametrize("stall_at", [0, 2, 9])
def test_decode_whose_loads_stop_gives_up(fmt, stall_at):
    # no weights arrive after a CTA's stall_at-th stage (of 15 or more): every wait behind them runs out,
    # the call ends with the timeout code, and the next call, on a zeroed workspace, is right
    T, k, E, H, I = 24, 4, 24, 2048, 1024
    g = torch.Generator(device=DEV).manual_seed(17)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF)  # noqa: E731
    gid = torch.from_numpy(np.random.default_rng(17).permuted(np.tile(np.arange(E, dtype=np.int32), (T, 1)), axis=1)
                           [:, :k].copy()).to(DEV)
    x, w1, w2 = rnd(T, H), 0.02 * rnd(E * 2 * I, H), 0.02 * rnd(E * H, I)
    sx = s1 = s2 = None
    if fmt is not None:
        (x, sx), (w1, s1), (w2, s2) = (pgg.mx_quantize_rowwise(x, fmt), pgg.mx_quantize_rowwise_blocked(w1, fmt),
                                       pgg.mx_quantize_rowwise_blocked(w2, fmt))
    ws = pgg.moe_decode_workspace(T, k, H, I, E, fmt)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call():
        if fmt is None:
            return pgg.moe_decode(x, gid, None, w1.view(E, 2 * I, H), w2.view(E, H, I), ws=ws, err=err)
        return pgg.mx_moe_decode(fmt, x, sx, gid, None, w1, s1, w2, s2, ws=ws, err=err)

    good = call()
    out = torch.zeros(T, H, dtype=BF, device=DEV)
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    torch.cuda.synchronize()
    t0 = time.monotonic()
    st = _binding.lib().pgg_test_stalled_moe_decode(
        {None: 0, "e4m3": 1, "e2m1": 2}[fmt], p(x), p(sx), p(gid), p(w1), p(s1), p(w2), p(s2), p(out), T, k, H, I, E,
        stall_at, 2_000_000, p(ws), ws.numel(), p(err), torch.cuda.current_stream().cuda_stream)
    assert st == 0 and pgg.read_error(err) == 17
    assert time.monotonic() - t0 < 5.0
    ws.zero_()
    err.zero_()
    assert torch.equal(call(), good) and pgg.read_error(err) == 0


def test_route_decode_equals_the_long_path():
    # route -> few-token layer against route -> permute -> grouped GEMMs -> combine
    rng = np.random.default_rng(15)
    T, k, E, H, I = 48, 4, 16, 256, 384
    x, gate = _bf(rng, T, H).to(DEV), _bf(rng, 1, E, H, scale=0.1).to(DEV)
    W1, W2 = _bf(rng, E, 2 * I, H, scale=0.06).to(DEV), _bf(rng, E, H, I, scale=0.05).to(DEV)
    one = torch.tensor([T], dtype=torch.int32, device=DEV)
    logits = pgg.grouped_gemm_fwd(x, gate, one)
    ids, w = pgg.moe_route(logits, k)
    out = pgg.moe_decode(x, ids, w, W1, W2)
    Xs, lens, pos = pgg.moe_permute(ids, x, E)
    A, _ = pgg.grouped_fc1_swiglu(Xs, W1, lens, save_h=False)
    ref = pgg.moe_combine(pgg.grouped_gemm_fwd(A, W2, lens), pos, w)
    # the long path rounds A and each expert's output to bf16
    util.assert_close(out, util.f64(ref), "few-token layer against the grouped GEMMs")
    rpos, rlens, _ = mg.permute(ids.cpu().numpy(), E)
    xs = mg.permute_rows(util.f64(x), rpos)
    a = og.swiglu_fwd(og.grouped_gemm_fwd(xs, util.f64(W1), rlens))
    exact = mg.combine(og.grouped_gemm_fwd(a, util.f64(W2), rlens), rpos, w.double().cpu().numpy())
    util.assert_close(out, exact, "few-token layer against the oracle's grouped GEMMs")
