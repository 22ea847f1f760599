"""The router's weights and gradient where scores leave fp32's range, against the 64-bit oracle.

Tolerances as for the other router tests: weights within 2^-18 of themselves, gradients within 2^-18
(fp32) or 2^-8 (bf16) of themselves plus 2^-18 or 2^-16 of the magnitudes that are summed."""
import numpy as np
import pytest
import torch

from oracle import block as ob

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _check(x, b, k, score, renormalize):
    ids, w = pgg.moe_route(x.to(DEV), k, None if b is None else b.to(DEV), score, renormalize, 2.5)
    z, bias = x.float().numpy(), None if b is None else b.numpy()
    rid, rw = ob.moe_route(z, bias, k, score, renormalize, 2.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    # (what is below fp32's range itself may come out as zero)
    np.testing.assert_array_less(np.abs(w.double().cpu().numpy() - rw), 2.0 ** -18 * np.abs(rw) + 1e-37)
    dw = torch.from_numpy(np.random.default_rng(k).standard_normal((len(x), k)).astype(np.float32))
    d = pgg.moe_route_bwd(x.to(DEV), ids, dw.to(DEV), None if b is None else b.to(DEV), score, renormalize, 2.5)
    ref = ob.moe_route_bwd(z, bias, rid, dw.double().numpy(), score, renormalize, 2.5)
    rel, tiny = (2.0 ** -8, 2.0 ** -16) if x.dtype == BF else (2.0 ** -18, 2.0 ** -18)
    mag = 2.5 * np.abs(dw.double().numpy()).sum(1, keepdims=True)
    np.testing.assert_array_less(np.abs(d.double().cpu().numpy() - ref), rel * np.abs(ref) + tiny * mag + 1e-37)
    return w, rw


@pytest.mark.parametrize("T", [3, 1027])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("low", [-59.0, -61.0, -87.0, -95.0, -104.0, -300.0, -690.0])
def test_sigmoid_scores_far_below(T, dtype, with_bias, low):
    # the sum of the chosen sigmoids is below fp32's range, their ratios are not
    rng = np.random.default_rng(7)
    x = torch.from_numpy((low - 3.0 * rng.random((T, 16))).astype(np.float32))
    b = None
    if with_bias:  # and the bias chooses them although others score higher
        x[:, ::2] = 2.0
        b = torch.zeros(16)
        b[::2] = -5000.0
    x = x.to(dtype)
    for renormalize in (True, False):
        w, rw = _check(x, b, 4, "sigmoid", renormalize)
    assert (rw < 1.0).all()
    w, rw = _check(x, b, 4, "sigmoid", True)
    np.testing.assert_allclose(w.double().cpu().numpy().sum(1), 2.5, rtol=1e-5)


@pytest.mark.parametrize("T", [2, 1026])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_sigmoid_scores_of_every_size(T, dtype):
    # choices in and far out of range side by side, masked ones, and a mask by the type's lowest value
    x = torch.tensor([[5.0, -20.0, -70.0, -200.0, -650.0, -float("inf"), 0.0, -1e4],
                      [-float("inf"), -80.0, -90.0, torch.finfo(dtype).min, -95.0, -1e4, -float("inf"), -120.0]])
    x = x.repeat(T // 2, 1).to(dtype)
    for k in (1, 3, 8):
        for renormalize in (True, False):
            _check(x, None, k, "sigmoid", renormalize)
            _check(x, torch.linspace(0, 50, 8), k, "sigmoid", renormalize)
    # one choice alone has the whole weight, however small its score
    w, _ = _check(x[:, 2:5].contiguous(), None, 1, "sigmoid", True)
    assert (w == 2.5).all()
