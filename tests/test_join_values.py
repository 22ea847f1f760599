"""The joint's gradients where a row's gate, its norm or one of its elements is not finite: what the mask drops passes nothing
on, to dx, to the sums over rows, to other rows.

An element that is dropped is 0 in the forward pass whatever it, its row's norm and its row's gate hold, so nothing depends
on it: the sums over rows have the bits that they have where that row's gradient is 0."""
import pytest
import torch

from oracle import linear as ol
from test_parity_join import BF, DEV, _bf

import numpy as np

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
SIZES = [(40, 264), (7, 1056), (90, 3200), (9, 4096), (41, 8264)]   # one and two pieces a thread, clusters


def _setup(R, C, p=0.5):
    rng = np.random.default_rng(C)
    x, dh = _bf(rng, R, C).to(DEV), _bf(rng, R, C).to(DEV)
    g1 = _bf(rng, C).to(DEV)
    state = torch.tensor([C, R], device=DEV)
    keep = torch.from_numpy(ol.keep(R, C, p, (C, R))).to(DEV)
    return rng, x, dh, g1, {"p": p, "rng": state}, keep


@pytest.mark.parametrize("R,C", SIZES)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_a_row_gate_without_a_value(R, C, value):
    rng, x, dh, g1, drop, keep = _setup(R, C)
    gate = torch.from_numpy(rng.standard_normal(R).astype(np.float32)).to(DEV)
    bad = gate.clone()
    rows = [1, R - 1]
    bad[rows] = value
    ref = pgg.block_join_bwd(None, dh, x, gate=gate, **drop)
    got = pgg.block_join_bwd(None, dh, x, gate=bad, **drop)
    others = torch.ones(R, dtype=torch.bool, device=DEV)
    others[rows] = False
    assert torch.equal(got[0][others], ref[0][others]) and torch.equal(got[1], ref[1])   # dx, dresidual
    assert (got[0][~keep] == 0).all()
    assert not torch.isfinite(got[0][rows][keep[rows] & (dh[rows] != 0)]).any()
    assert torch.equal(got[4], ref[4])   # a gate's own gradient does not read it
    # with the norm of x: its weight's gradient in the columns that the rows drop
    rstd = torch.rsqrt(x.float().square().mean(1) + 1e-6)
    d0 = dh.clone()
    d0[rows] = 0
    ref = pgg.block_join_bwd(None, d0, x, None, rstd, gamma_post=g1, gate=gate, **drop)
    got = pgg.block_join_bwd(None, dh, x, None, rstd, gamma_post=g1, gate=bad, **drop)
    free = ~keep[rows].any(0)
    assert free.any() and torch.equal(got[2][free], ref[2][free])
    assert not torch.isfinite(got[2][~free]).any()
    assert torch.equal(got[0][others], ref[0][others])


@pytest.mark.parametrize("R,C", SIZES)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("gate", [None, "row", "column"])
def test_a_row_without_a_norm(R, C, value, gate):
    rng, x, dh, g1, drop, keep = _setup(R, C)
    gate = {None: None, "row": torch.rand(R, generator=torch.Generator().manual_seed(1)).to(DEV),
            "column": _bf(rng, C).to(DEV)}[gate]
    bad = x.clone()
    row = R // 2
    kept, dropped = keep[row].nonzero()[0].item(), (~keep[row]).nonzero()[0].item()
    for col in (kept, dropped):
        bad[row, col] = value
        norm = lambda t: torch.rsqrt(t.float().square().mean(1) + 1e-6)  # noqa: E731
        d0 = dh.clone()
        d0[row] = 0
        ref = pgg.block_join_bwd(None, d0, x, None, norm(x), gamma_post=g1, gate=gate, **drop)
        got = pgg.block_join_bwd(None, dh, bad, None, norm(bad), gamma_post=g1, gate=gate, **drop)
        others = torch.arange(R, device=DEV) != row
        assert torch.equal(got[0][others], ref[0][others])
        free = ~keep[row]
        assert torch.equal(got[2][free], ref[2][free])
        if gate is not None and gate.dtype == BF:
            assert torch.equal(got[4][free], ref[4][free])
        bad[row, col] = x[row, col]


@pytest.mark.parametrize("R,C", SIZES)
def test_dropped_elements_pass_nothing_on(R, C):
    # no norm of x: NaN and infinities in every dropped place change no bit of any gradient
    rng, x, dh, g1, drop, keep = _setup(R, C)
    gate = _bf(rng, C).to(DEV)
    bad = torch.where(keep, x, torch.where(torch.arange(C, device=DEV) % 2 == 0, NAN, INF).to(BF))
    for kw in ({"gate": gate}, {}, {"gate": torch.ones(R, device=DEV)}):
        ref, got = (pgg.block_join_bwd(None, dh, t, **kw, **drop) for t in (x, bad))
        assert all(torch.equal(a, b) for a, b in zip(ref, got) if a is not None)
