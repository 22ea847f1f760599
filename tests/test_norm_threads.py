"""The norm's backward called from several host threads, each on its own stream."""
import sys
import threading

import pytest
import torch

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _inputs(C, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF)  # noqa: E731
    h = rnd(8, C)
    return rnd(8, C), rnd(8, C), h, rnd(C), torch.rsqrt(h.float().square().mean(1) + 1e-6)


@pytest.mark.parametrize("wide,narrow", [(8192, 3136), (16384, 8256)])
def test_norm_bwd_widths_of_one_kernel_from_many_threads(wide, narrow):
    # two widths that one kernel serves with different amounts of shared memory
    call = pgg.lib().pgg_add_rmsnorm_bwd
    ref = {C: pgg.add_rmsnorm_bwd(*_inputs(C, C)) for C in (wide, narrow)}
    bad = []

    def work(C):
        a = _inputs(C, C)
        dx, dg = torch.empty_like(a[0]), torch.empty(C, device=DEV)
        ws = torch.empty(pgg.add_rmsnorm_bwd_workspace_size(8, C), dtype=torch.uint8, device=DEV)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        args = (*(t.data_ptr() for t in a), 8, C, dx.data_ptr(), dg.data_ptr(), ws.data_ptr(), ws.numel(), s.cuda_stream)
        failed = 0
        for i in range(10000):
            failed += call(*args) != 0
            if i % 200 == 199:
                s.synchronize()
        if failed or not (torch.equal(dx, ref[C][0]) and torch.equal(dg, ref[C][1])):
            bad.append((C, failed))

    switch = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=work, args=(C,)) for C in (wide, narrow) * 3]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(switch)
    assert not bad
