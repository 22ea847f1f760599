"""The few-token layer on inputs whose sums are exact, so that a lost or doubled term shows.

Every gate sum is 32 (silu(32) is 32 in fp32), every up sum a value of the e2m1 grid with a 6 in
each block of 32, so that the activation's MX codes have nothing to round; weights, inputs and the
products' sums are small whole numbers.  Every 64-wide piece of the reduction holds a term of each
sum, and terms cancel between pieces, so a piece that is left out or added twice changes the result.

So an output is the sum rounded to bf16, up to silu's few ulp of fp32: it lies between the roundings
of the sum less and plus 2^-20 of the terms' magnitudes."""
import numpy as np
import pytest
import torch

from oracle import block as ob

DEV = "cuda"
BF = torch.bfloat16
GRID = np.array([1, 2, 3, 4, 6, -1, -2, -3, -4, -6], dtype=np.float32)
# two numbers of the grid with a given sum on the grid
PAIRS = {v: [(a, b) for a in GRID for b in GRID if a + b == v] for v in GRID}
KINDS = 4  # tokens t, t + KINDS, ... have the same inputs


def _sums(rng, v, pieces):
    """Terms [pieces, ...] on the grid that add up to v [...]: +r, -r in pairs, and v in what is left."""
    out = np.zeros((pieces, *v.shape), dtype=np.float32)
    order = rng.permutation(pieces)
    n = 1 if pieces % 2 else 2
    for i in range(n, pieces, 2):
        r = rng.choice(GRID, size=v.shape)
        out[order[i]], out[order[i + 1]] = r, -r
    if n == 1:
        out[order[0]] = v
    else:
        for g in GRID:
            pick = np.array(PAIRS[g], dtype=np.float32)[rng.integers(len(PAIRS[g]), size=v.shape)]
            for i in range(2):
                out[order[i]] = np.where(v == g, pick[..., i], out[order[i]])
    return out


def _layer(T, k, E, H, I, seed, common=None, ids=None):
    """-> ids, w, x, W1, W2 (float32, exact in every format), the result and its terms' magnitudes."""
    rng = np.random.default_rng([seed, T, k, E, H, I])
    pieces = -(-H // 64)
    cols = np.stack([64 * p + rng.permutation(min(64, H - 64 * p))[:1 + KINDS] for p in range(pieces)])
    v = rng.choice(GRID, size=(E, I, KINDS))
    for b in range(0, I, 32):  # a six in every block, whatever the kind
        v[:, b + rng.integers(min(32, I - b))] = 6 * rng.choice([-1.0, 1.0], size=(E, KINDS))
    W1 = np.zeros((E, 2 * I, H), dtype=np.float32)
    gate = _sums(rng, np.full((E, I), 4.0, dtype=np.float32), pieces) * 8
    for p in range(pieces):
        W1[:, :I, cols[p, 0]] = gate[p]
    for q in range(KINDS):
        up = _sums(rng, v[..., q], pieces)
        for p in range(pieces):
            W1[:, I:, cols[p, 1 + q]] = up[p]
    x = np.zeros((T, H), dtype=np.float32)
    x[:, cols[:, 0]] = 1
    for t in range(T):
        x[t, cols[:, 1 + t % KINDS]] = 1
    W2 = rng.choice(GRID, size=(E, H, I))
    if ids is None:
        ids = rng.integers(E, size=(T, k)).astype(np.int32)  # repeats: their weights add up
        if common is not None:
            ids[:, rng.integers(k)] = common
    w = rng.choice([0.25, 0.5, 1.0], size=(T, k)).astype(np.float32)
    ref, mag = np.zeros((T, H)), np.zeros((T, H))
    for q in range(KINDS):
        a = 32 * v[..., q].astype(np.float64)
        y, m = np.einsum("ehi,ei->eh", W2, a), np.einsum("ehi,ei->eh", np.abs(W2), np.abs(a))
        for t in range(q, T, KINDS):
            ref[t] = (w[t, :, None] * y[ids[t]]).sum(0)
            mag[t] = (w[t, :, None] * m[ids[t]]).sum(0)
    return ids, w, x, W1, W2, ref, mag


@pytest.mark.parametrize("H,I", [(128, 128), (320, 128), (1024, 64)])
def test_inputs_are_what_they_are_meant_to_be(H, I):
    ids, w, x, W1, W2, ref, mag = _layer(9, 3, 3, H, I, 0)
    for fmt in (None, "e4m3", "e2m1"):
        out, _, m = ob.moe_decode(x.astype(np.float64), ids, w, W1.astype(np.float64), W2.astype(np.float64), None, fmt)
        assert np.all(np.abs(out - ref) <= 1e-11 * mag)
    for t in (x, W1.reshape(-1, H), W2.reshape(-1, I)):  # on the coarsest format's grid
        b = t.reshape(len(t), -1, 32)
        e = np.floor(np.log2(np.maximum(np.abs(b).max(-1, keepdims=True), 1e-9))) - 2
        assert np.isin(np.abs(b) / 2.0 ** e, [0, 0.5, 1, 1.5, 2, 3, 4, 6]).all()


def _run(fmt, ids, w, x, W1, W2, times=1):
    import precision_grouped_gemm_gb300 as pgg
    E, H, I = W2.shape
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    X, U, V = d(x).to(BF), d(W1).to(BF), d(W2).to(BF)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if fmt is None:
        ws = pgg.moe_decode_workspace(*ids.shape, H, I, E)
        outs = [pgg.moe_decode(X, d(ids), d(w), U, V, ws=ws, err=err) for _ in range(times)]
    else:
        ws = pgg.moe_decode_workspace(*ids.shape, H, I, E, fmt)
        a = (fmt, *pgg.mx_quantize_rowwise(X, fmt), d(ids), d(w),
             *pgg.mx_quantize_rowwise_blocked(U.view(-1, H), fmt), *pgg.mx_quantize_rowwise_blocked(V.view(-1, I), fmt))
        outs = [pgg.mx_moe_decode(*a, ws=ws, err=err) for _ in range(times)]
    assert pgg.read_error(err) == 0
    assert not ws[1024:1024 + 160 * 128 * 512 * 4].any()  # the partial sums' places are clear again
    return outs


def _check(outs, ref, mag):
    lo, hi = (torch.from_numpy(ref + s * 2.0 ** -20 * mag).to(BF).double().numpy() for s in (-1, 1))
    for o in outs:
        got = o.double().cpu().numpy()
        bad = ~((lo <= got) & (got <= hi))
        assert not bad.any(), f"{bad.sum()} of {bad.size}, e.g. {got[bad][:4]} for {ref[bad][:4]}"
        assert torch.equal(o, outs[0])


# Few (expert, tile)s and a long reduction: each is divided over up to 64 CTAs, one stage each, whose
# sums the first one adds to its own, one after the other.
CHAINS = [(1, 1, 1, 2048, 384), (1, 1, 1, 4096, 128), (2, 2, 2, 1024, 256), (5, 1, 1, 4096, 256), (8, 2, 2, 2048, 128),
          (12, 1, 1, 2048, 256), (33, 1, 1, 2048, 128), (100, 1, 1, 1280, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [None, "e4m3", "e2m1"])
@pytest.mark.parametrize("T,k,E,H,I", CHAINS)
def test_tile_divided_over_many_ctas(T, k, E, H, I, fmt):
    ids, w, x, W1, W2, ref, mag = _layer(T, k, E, H, I, 1)
    _check(_run(fmt, ids, w, x, W1, W2, times=20), ref, mag)


# Every token names one common expert, so its MMAs have up to 128 columns (256 for the two bf16 parts of
# the activation): one accumulator instead of two, all four words of a scale atom's rows, and with k = 32
# the least shared memory for the ring (two stages in bf16).
FULL = [(128, 1, 1, 512, 384), (128, 1, 2, 384, 128), (128, 2, 2, 640, 256), (128, 8, 16, 384, 384),
        (128, 32, 40, 256, 256), (113, 8, 12, 512, 128), (100, 4, 8, 384, 640), (97, 3, 3, 1152, 384)]


def _common(T, k, E, H, I):
    return _layer(T, k, E, H, I, 2, common=E - 1)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [None, "e4m3", "e2m1"])
@pytest.mark.parametrize("T,k,E,H,I", FULL)
def test_an_expert_that_every_token_names(T, k, E, H, I, fmt):
    ids, w, x, W1, W2, ref, mag = _common(T, k, E, H, I)
    assert (ids == E - 1).any(1).all()
    _check(_run(fmt, ids, w, x, W1, W2, times=3), ref, mag)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,H,I", [(128, 1, 1, 520, 200), (128, 8, 16, 72, 264), (128, 32, 40, 328, 136),
                                       (120, 2, 5, 1032, 72), (128, 3, 3, 8, 1000)])
def test_an_expert_that_every_token_names_off_the_tiles(T, k, E, H, I):
    ids, w, x, W1, W2, ref, mag = _common(T, k, E, H, I)
    _check(_run(None, ids, w, x, W1, W2, times=3), ref, mag)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [None, "e4m3", "e2m1"])
def test_weights_past_32_bit_offsets(fmt):
    # 1024 experts of 2048 x 1152: 4.8 G elements of W1 and 2.4 G of W2.  The tokens name the experts
    # at both ends, just below and above an element offset of 2^31 and 2^32, and around byte offsets of those.
    import precision_grouped_gemm_gb300 as pgg
    E, H, I = 1024, 2048, 1152
    per1, per2 = 2 * I * H, H * I
    at = {0, E - 1}
    for n in (2 ** 31, 2 ** 32):
        for size in {None: 2, "e4m3": 1, "e2m1": 0.5}[fmt], 1:  # in bytes, in elements
            for per in (per1, per2):
                e = int(n / size / per)
                at |= {e - 1, e, e + 1}
    named = np.array(sorted(e for e in at if e < E), dtype=np.int32)
    T = len(named)
    some, w, x, W1, W2, ref, mag = _layer(T, 2, T, H, I, 3, ids=np.stack([np.arange(T), np.arange(T)[::-1]], 1).astype(np.int32))
    ids, d = torch.from_numpy(named[some]).to(DEV), lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    X, where = d(x).to(BF), d(named).long()
    if fmt is None:
        U = torch.full((E, 2 * I, H), float("nan"), dtype=BF, device=DEV)  # no other expert has a part
        V = torch.full((E, H, I), float("nan"), dtype=BF, device=DEV)
        U[where], V[where] = d(W1).to(BF), d(W2).to(BF)
        out = pgg.moe_decode(X, ids, d(w), U, V)
    else:
        def spread(m, rows, cols):  # codes and blocked scales (whole atoms of 128 rows) of the named experts
            c, s = pgg.mx_quantize_rowwise_blocked(d(m).to(BF).view(-1, cols), fmt)
            c, s = c.view(T, -1), s.view(T, -1)
            C = torch.empty((E, c.shape[1]), dtype=torch.uint8, device=DEV)
            S = torch.full((E, s.shape[1]), 255, dtype=torch.uint8, device=DEV)  # NaN scales elsewhere
            C[where], S[where] = c, s
            return C.view(E * rows, -1), S.view(E * rows, -1)
        out = pgg.mx_moe_decode(fmt, *pgg.mx_quantize_rowwise(X, fmt), ids, d(w), *spread(W1, 2 * I, H), *spread(W2, H, I))
    _check([out], ref, mag)
