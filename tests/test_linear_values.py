"""The activations of grouped_linear and their derivatives over the whole range of their arguments, one value at a
time: tails, numbers whose product with alpha passes fp32's range, infinities and NaN.

The forward pass gets z exactly: z is the sum of two bf16 numbers, multiplied by ones (K = 8, the rest zeros).  The
derivative in fp32 is the biases' gradient of groups of one row.

Tolerances, u = 2^-24, from the arithmetic.  An exponential of -x: the argument alpha v is rounded, x u; the full one has 2
units, 4 u, the short one 2 + 1.173 x units, (4 + 2.4 x) u, by their documented bounds: at most (4 + 3.4 x) u.  A sigmoid is
1 / (1 + e) or e / (1 + e): sum and quotient (two units) 5 u, a product u, and the exponential's error times its share
sigmoid(-v): (10 + 3.4 |v| sigmoid(-v)) u.  1 - s has the error of s and u, which a derivative multiplies by |v| s.  Phi(-|z|): the exponential's argument z^2 / 2 is rounded, z^2 u; the fit 1.7e-7 = 3 u; its variable 5 u, to which the fit's
relative slope is 2.7 at most; its own eight steps 4 u: 24 u + z^2 u, twice the last with the short exponential.  A product
after that is u each.  A number below 2^-126 is off by 2^-149 (a rounding there is half of that, the short exponential's
flush of its last bit one), times what it is multiplied with; the fp32 result itself by 2^-149 too.  bf16 results add
half a step, 2^-8."""
import numpy as np
import pytest
import torch

from oracle import linear as ol
import util

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
BIG = 3.0e38
ALPHAS = (1.0, 1.702, -0.7, 1e30, 1e-30)


def _grid(n=2048):
    """bf16 numbers: dense to +-15, then by powers to the largest, both signs, and zeros."""
    near = torch.linspace(-15, 15, n).to(BF).double()
    far = torch.logspace(-38, 38, 305, dtype=torch.float64).to(BF).double()
    return torch.cat((near, far, -far, torch.tensor([0.0, BIG, -BIG], dtype=torch.float64).to(BF).double()))


def _sig(v):
    return np.vectorize(ol._sigmoid, otypes=[float])(v)


def _forward(z, act, out, extra=None, **form):
    """act of the numbers z = hi + lo (both bf16), a row each; extra: the other half's numbers."""
    z = z.double()
    hi = z.to(BF)
    lo = (z - hi.double()).to(BF)
    assert torch.equal(hi.double() + lo.double(), z)
    X = torch.zeros(len(z), 8, dtype=BF)
    X[:, 0], X[:, 1] = hi, lo
    n = 16 if act == "swiglu" else 8
    W = torch.zeros(n, 8, dtype=BF)
    W[:, :2] = 1
    if extra is not None:
        X[:, 2] = extra.to(BF)
        W[n // 2:] = 0
        W[n // 2:, 2] = 1
    Y, _ = pgg.grouped_linear(X.to(DEV), W.to(DEV), act=act, out_dtype=out, **form)
    assert all(torch.equal(Y[:, 0].nan_to_num(7), Y[:, i].nan_to_num(7)) for i in range(1, Y.shape[1]))
    return Y[:, 0].double().cpu().numpy()


def _near(got, ref, rel, absolute, out, what):
    bound = rel * np.abs(ref) + absolute + (2.0 ** -8 * np.abs(ref) + 2.0 ** -134 if out == BF else 2.0 ** -149)
    err = np.abs(got - ref)
    bad = ~((err <= bound) | (got == ref))
    assert not bad.any(), (what, bad.sum(), got[bad][:4], ref[bad][:4], (err / bound)[bad].max())


def _fine():
    """Numbers of 16 bits to +-13."""
    hi = torch.linspace(-13, 13, 1999).to(BF).double()
    return hi + (hi * 2.0 ** -9 * 0.7).to(BF).double()


@pytest.mark.parametrize("out", [BF, F32])
def test_gelu_in_its_tails(out):
    for z in (_grid(), _fine()):
        v = z.numpy()
        rel = (28 + v * v * (2 if out == BF else 1)) * U
        # (past the range of the exponential the value is below it)
        far = np.abs(v) > 14
        _near(_forward(z, "gelu", out), ol.act(v[:, None], "gelu")[:, 0], np.where(far, 4 * U, rel),
              (np.abs(v) + 1) * 2.0 ** -148, out, "gelu")


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("alpha", ALPHAS)
def test_silu_in_its_tails(alpha, out):
    for z in (_grid(), _fine()):
        v = z.numpy()
        a = alpha * v
        rel = (12 + 3.4 * np.minimum(np.abs(a), 104) * _sig(-a)) * U
        # (1 + e^-v above 2^126 gives 0, where the sigmoid is below 2^-126)
        _near(_forward(z, "silu", out, alpha=alpha), ol.act(v[:, None], "silu", alpha)[:, 0], rel, np.abs(v) * 2.0 ** -125,
              out, "silu")


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("alpha", ALPHAS)
def test_swiglu_in_its_tails(alpha, out):
    z = _grid()
    u = torch.tensor([0.5, -1.25, 3.0, -7.0] * (len(z) // 4 + 1))[:len(z)].double()
    for offset, limit in ((0.0, 0.0), (1.0, 7.0), (1.0, 2.5)):
        v, w = z.numpy(), u.numpy()
        ref = ol.act(np.stack([v, w], 1), "swiglu", alpha, offset, limit)[:, 0]
        g = np.minimum(v, limit) if limit else v
        a = alpha * g
        rel = (14 + 3.4 * np.minimum(np.abs(a), 104) * _sig(-a)) * U
        got = _forward(z, "swiglu", out, u, alpha=alpha, offset=offset, limit=limit)
        ok = np.abs(ref) < 3e38   # (past that the result is infinite)
        assert np.array_equal(np.isinf(got[~ok]), np.abs(ref[~ok]) > 3.5e38) or (np.abs(ref[~ok]) < 3.5e38).any()
        _near(got[ok], ref[ok], rel[ok], 8 * (np.abs(g[ok]) * 2.0 ** -125 + 2.0 ** -149), out, "swiglu")  # |u + offset| <= 8


# ---------------------------------------------------------------- derivatives

def _slope(z, act, u=None, dy=1.0, **form):
    """(the bf16 dZ, the fp32 ones) of rows of their own groups: [n, N]."""
    n = len(z)
    gl = torch.ones(1024, dtype=torch.int32)
    N = 16
    Z = torch.zeros(-(-n // 1024) * 1024, N, dtype=BF)
    if act == "swiglu":
        Z[:n, :8], Z[:n, 8:] = z.to(BF)[:, None], u.to(BF)[:, None]
    else:
        Z[:n] = z.to(BF)[:, None]
    dY = torch.full((len(Z), 8 if act == "swiglu" else 16), dy, dtype=BF, device=DEV)
    dz, db = [], []
    for i in range(0, len(Z), 1024):
        a, b = pgg.grouped_linear_bwd(dY[i:i + 1024], Z[i:i + 1024].to(DEV), gl.to(DEV), act=act, **form)
        dz.append(a)
        db.append(b)
    return torch.cat(dz)[:n].double().cpu().numpy(), torch.cat(db)[:n].double().cpu().numpy()


def _terms(a):
    """Bound of s + a s (1 - s), s = sigmoid(a): the sigmoid's error, the complement's, four products and the sum."""
    s, c = _sig(a), _sig(-a)
    m = np.minimum(np.abs(a), 104)
    e = (10 + 3.4 * m * c) * s
    return (e + m * s * (e + 1) + m * c * (e + 1) + 4 * (s + m * s * c)) * U + 2.0 ** -125


@pytest.mark.parametrize("alpha", ALPHAS)
def test_silu_slope_in_its_tails(alpha):
    z = _grid()
    v = z.numpy()
    ref = ol.act_bwd(np.ones((len(v), 1)), v[:, None], "silu", alpha)
    dz, db = _slope(z, "silu", alpha=alpha)
    bound = (_terms(alpha * v) + abs(alpha) * 2.0 ** -148)[:, None]   # (alpha times two products)
    _near(db, np.repeat(ref, 16, 1), 0.0, bound, F32, "dbias")
    _near(dz, np.repeat(ref, 16, 1), 0.0, bound, BF, "dZ")


def test_gelu_slope_in_its_tails():
    z = _grid()
    v = z.numpy()
    ref = np.repeat(ol.act_bwd(np.ones((len(v), 1)), np.clip(v, -40, 40)[:, None], "gelu"), 16, 1)
    dz, db = _slope(z, "gelu")
    w = np.minimum(np.abs(v), 20)
    e = np.exp(-w * w / 2)
    bound = ((28 + 2 * w * w) * (0.5 * e + 0.4 * w * e) + 2) * U + 2.0 ** -125
    _near(db, ref, 0.0, bound[:, None], F32, "dbias")
    _near(dz, ref, 0.0, bound[:, None], BF, "dZ")


@pytest.mark.parametrize("alpha", ALPHAS)
@pytest.mark.parametrize("offset,limit", [(0.0, 0.0), (1.0, 7.0)])
def test_swiglu_slope_in_its_tails(alpha, offset, limit):
    z = _grid()
    u = torch.tensor([0.5, -1.25, 3.0, -8.0] * (len(z) // 4 + 1))[:len(z)].double()
    v, w = z.numpy(), u.numpy()
    ref = ol.act_bwd(np.ones((len(v), 1)), np.stack([v, w], 1), "swiglu", alpha, offset, limit)
    g = np.minimum(v, limit) if limit else v
    up = np.abs((np.clip(w, -limit, limit) if limit else w) + offset)
    dz, db = _slope(z, "swiglu", u, alpha=alpha, offset=offset, limit=limit)
    a = alpha * g
    b_g = (_terms(a) + abs(alpha) * 2.0 ** -148) * up
    b_u = (13 + 3.4 * np.minimum(np.abs(a), 104) * _sig(-a)) * U * np.abs(ref[:, 1]) + np.abs(g) * 2.0 ** -125 + 2.0 ** -149
    for got, out in ((db, F32), (dz, BF)):
        _near(got[:, 0], ref[:, 0], 0.0, b_g, out, "dg")
        _near(got[:, 8], ref[:, 1], 0.0, b_u, out, "du")


# ---------------------------------------------------------------- infinities and NaN

def test_special_values_through_the_activations():
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([inf, -inf, nan, 1.0], dtype=BF, device=DEV)
    X = torch.zeros(4, 8, dtype=BF, device=DEV)
    W = torch.zeros(8, 8, dtype=BF, device=DEV)
    bias = torch.zeros(4, 8, dtype=BF, device=DEV) + z[:, None]
    gl = torch.ones(4, dtype=torch.int32, device=DEV)
    for out in (BF, F32):
        for act in ("silu", "gelu"):
            Y, Z = pgg.grouped_linear(X, W.expand(4, 8, 8).contiguous(), gl, bias=bias, act=act, save_z=True, out_dtype=out)
            assert torch.equal(Z.nan_to_num(5.0, 6.0, 7.0), (torch.zeros_like(Z) + z[:, None]).nan_to_num(5.0, 6.0, 7.0))
            # (the value at -inf is -inf times 0)
            assert (Y[0] == inf).all() and torch.isnan(Y[1]).all() and torch.isnan(Y[2]).all() and torch.isfinite(Y[3]).all()
        W2, b2 = torch.zeros(4, 16, 8, dtype=BF, device=DEV), torch.ones(4, 16, dtype=BF, device=DEV)
        for side in (0, 1):
            b = b2.clone()
            b[:, 8 * side:8 * side + 8] = z[:, None]
            Y, _ = pgg.grouped_linear(X, W2, gl, bias=b, act="swiglu", limit=2.0, out_dtype=out)
            v = b.double().cpu().numpy()
            ref = ol.act(v[[3]], "swiglu", 1.0, 0.0, 2.0)
            assert np.allclose(Y[3].double().cpu().numpy(), ref[0], rtol=2.0 ** -7)
            # (clamped: inf is 2, -inf of the up half -2; of the gate's -inf the limit stays -inf, times 0)
            assert torch.isfinite(Y[0]).all() and torch.isnan(Y[2]).all()
            assert torch.isnan(Y[1]).all() if side == 0 else torch.isfinite(Y[1]).all()


@pytest.mark.parametrize("lens", [[3, 0, 5, 1, 40], [600, 0, 700, 129, 300]])
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", None])
def test_a_row_without_a_value_stays_in_its_group_and_column(act, lens):
    """NaN and infinities in one row's columns: the other groups' sums, columns and rows keep their bits."""
    M, N = sum(lens), 528
    g = torch.Generator().manual_seed(3)
    Z = torch.randn(M, N, generator=g).to(BF).to(DEV)
    dY = torch.randn(M, N // 2 if act == "swiglu" else N, generator=g).to(BF).to(DEV)
    gl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    run = lambda y, z: pgg.grouped_linear_bwd(y, z if act else None, gl, act=act)  # noqa: E731
    dz, db = run(dY, Z)
    row = lens[0] + 2   # of group 2
    y2 = dY.clone()
    y2[row, 5], y2[row, 9], y2[row, 200] = float("nan"), float("inf"), float("-inf")
    dz2, db2 = run(y2, Z)
    cols = [5, 9, 200]
    hit = torch.zeros_like(db, dtype=torch.bool)
    for c in cols + [c + N // 2 for c in cols if act == "swiglu"]:
        hit[2, c] = True
    assert not torch.isfinite(db2[hit]).any() and torch.equal(db2[~hit], db[~hit])
    if act:
        at = torch.zeros_like(dz, dtype=torch.bool)
        at[row] = hit[2]
        assert not torch.isfinite(dz2[at]).any() and torch.equal(dz2[~at], dz[~at])
        z2 = Z.clone()
        z2[row, 5] = float("nan")
        dz3, db3 = run(dY, z2)
        hit = torch.zeros_like(db, dtype=torch.bool)
        hit[2, 5] = True
        if act == "swiglu":
            hit[2, 5 + N // 2] = True
        at = torch.zeros_like(dz, dtype=torch.bool)
        at[row] = hit[2]
        assert torch.isnan(db3[hit]).all() and torch.equal(db3[~hit], db[~hit])
        assert torch.isnan(dz3[at]).all() and torch.equal(dz3[~at], dz[~at])
