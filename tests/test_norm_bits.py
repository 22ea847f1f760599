"""The norm's outputs bit for bit, from its own rstd.

s = x + residual and y = (s rstd) gamma are one fp32 addition and two fp32 products an element, which
numpy does alike: h, y and the MX codes are then roundings of known numbers and have to be equal."""
import numpy as np
import pytest
import torch

from oracle import mx as omx

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.mark.parametrize("R,C", [(1, 32), (3, 96), (5, 1056), (2, 16384), (700, 288), (1300, 2048), (3, 8224)])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_norm_bits(R, C, residual, fmt):
    rng = np.random.default_rng([R, C, residual])
    t = lambda *s, scale=1.0: torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).to(BF)  # noqa: E731
    x, g = t(R, C), 1 + t(C, scale=0.3)
    r = t(R, C, scale=3.0) if residual else None
    x[:, C // 2:C // 2 + 32] *= 2.0 ** -20    # blocks far below the others, and one of zeros
    if r is not None:
        r[:, C // 2:C // 2 + 32] *= 2.0 ** -20
    x[R - 1, :32] = 0
    if r is not None:
        r[R - 1, :32] = 0
    h, y, codes, scales, rstd = pgg.add_rmsnorm(x.to(DEV), None if r is None else r.to(DEV), g.to(DEV), 1e-5, fmt=fmt)
    s = x.float().numpy() if r is None else x.float().numpy() + r.float().numpy()
    row = (s * rstd.cpu().numpy()[:, None]) * g.float().numpy()[None, :]
    assert row.dtype == np.float32
    assert torch.equal(h.cpu(), torch.from_numpy(s).to(BF)) and torch.equal(y.cpu(), torch.from_numpy(row).to(BF))
    rs, rc = omx.quantize_blocks(fmt, row.astype(np.float64).reshape(R, C // 32, 32))
    got = codes.cpu().numpy()
    got = omx.unpack_e2m1(got) if fmt == "e2m1" else got
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(got.reshape(rc.shape), rc)
