"""Calls of the few-token layer on several streams at once, each with its own workspace."""
import pytest
import torch

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def test_calls_that_overlap():
    E, H, I, k = 16, 512, 256, 4
    g = torch.Generator(device=DEV).manual_seed(1)
    rnd = lambda *s, scale=1.0: (scale * torch.randn(s, generator=g, device=DEV)).to(BF)  # noqa: E731
    W1, W2 = rnd(E, 2 * I, H, scale=H ** -0.5), rnd(E, H, I, scale=I ** -0.5)
    mx = [(*pgg.mx_quantize_rowwise_blocked(W1.view(-1, H), f), *pgg.mx_quantize_rowwise_blocked(W2.view(-1, I), f))
          for f in ("e4m3", "e2m1")]
    calls = []
    for T, fmt in ((1, None), (7, "e4m3"), (40, "e2m1"), (128, None)):
        x, ids = rnd(T, H), torch.randint(E, (T, k), generator=g, device=DEV, dtype=torch.int32)
        w, ws = torch.rand(T, k, generator=g, device=DEV), pgg.moe_decode_workspace(T, k, H, I, E, fmt)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        if fmt is None:
            f = lambda s, a=(x, ids, w, W1, W2), ws=ws, err=err: pgg.moe_decode(*a, ws=ws, err=err, stream=s)  # noqa: E731
        else:
            a = (fmt, *pgg.mx_quantize_rowwise(x, fmt), ids, w, *mx[fmt == "e2m1"])
            f = lambda s, a=a, ws=ws, err=err: pgg.mx_moe_decode(*a, ws=ws, err=err, stream=s)  # noqa: E731
        calls.append((f, err, f(None)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[f(s) for (f, _, _), s in zip(calls, streams)] for _ in range(50)]
    torch.cuda.synchronize()
    for i, (_, err, first) in enumerate(calls):
        assert pgg.read_error(err) == 0
        assert all(torch.equal(o[i], first) for o in outs)
