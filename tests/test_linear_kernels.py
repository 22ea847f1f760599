"""Every kernel of grouped_linear by name: the sizes that each is taken for, and each one's results, failure and
overlap at sizes of the tests' choice, whatever the sizes alone would take.

Tolerances: those derived in test_parity_linear.py, whose checks are used here."""
import ctypes

import numpy as np
import pytest
import torch

import test_parity_linear as tl
import util

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
ACTS = {None: 0, "silu": 1, "gelu": 2, "swiglu": 3}
SPLIT, ONE, PAIR = 0, 1, 2
INVALID = 1


def _plan(M, N, K, G=1, grouped=False, act=None, out=BF, sms=0):
    p = (ctypes.c_int32 * 4)()
    st = pgg.lib().pgg_test_linear_plan(M, N, K, G, int(grouped), ACTS[act], int(out == BF), sms, p)
    return st, tuple(p)


def _run(plan, X, W, lens, Y, bias=None, residual=None, act=None, Z=None, err=None, stall_at=-1, wait_ns=0, **form):
    """The call with that kernel -> its status; without act's numbers, the tests' own."""
    f = form or tl.FORMS[act]
    a = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    M, K = X.shape
    G, N, _ = W.shape
    return pgg.lib().pgg_test_planned_linear(
        *plan, a(X), a(W), a(lens), a(bias), a(residual), a(Y), int(Y.dtype == BF), a(Z), M, N, K, G, ACTS[act],
        f.get("alpha", 1.0), f.get("offset", 0.0), f.get("limit", 0.0), stall_at, wait_ns, a(err),
        torch.cuda.current_stream().cuda_stream)


# ---------------------------------------------------------------- the hooks' own refusals (no GPU)

def test_plan_refusals():
    from precision_grouped_gemm_gb300 import build
    build.build()
    for kw in ({"M": 0}, {"G": 0}, {"G": 2}, {"N": 4}, {"K": 4}, {"sms": -1}):
        st, _ = _plan(**{"M": 8, "N": 64, "K": 64, **kw})
        assert st == INVALID, kw
    assert _plan(8, 68, 64)[0] == 3 and _plan(8, 72, 64, act="swiglu")[0] == 3
    assert pgg.lib().pgg_test_linear_plan(8, 64, 64, 1, 0, 0, 1, 0, None) == INVALID
    P = 1 << 20
    run = lambda kind=1, at=-1, ns=0: pgg.lib().pgg_test_planned_linear(  # noqa: E731
        kind, 32, 1, P, P, P, P, P, P, 1, P, 8, 64, 64, 2, 0, 1.0, 0.0, 0.0, at, ns, None, None)
    assert run(kind=-1) == INVALID and run(kind=3) == INVALID and run(at=-2) == INVALID
    assert run(ns=50_000) == INVALID and run(ns=2_000_000_000) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="asks a machine without a device")
def test_no_plan_where_the_device_does_not_answer():
    # the clusters that fit are asked of the device: an answer that fails is the call's, not taken as one cluster
    from precision_grouped_gemm_gb300 import build
    build.build()
    for _ in range(2):
        assert _plan(1, 4096, 4096, sms=152)[0] not in (0, INVALID)
    assert _plan(4096, 2048, 72, sms=152)[0] == 0   # (too short to cut: nothing to ask)


# ---------------------------------------------------------------- what the sizes take

@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,G,act,out,plan", [
    # one row, a gate, a decode batch
    (1, 4096, 4096, 1, None, BF, (SPLIT, 16, 4, 1)), (37, 256, 4096, 1, None, F32, (SPLIT, 16, 8, 1)),
    (64, 4096, 4096, 1, None, BF, (SPLIT, 32, 2, 1)), (256, 1024, 4096, 1, None, BF, (SPLIT, 64, 4, 1)),
    (3219, 192, 6704, 1, None, BF, (SPLIT, 128, 2, 1)), (128, 5760, 2880, 32, "swiglu", BF, (ONE, 32, 1, 1)),
    # many short groups; fp32 results
    (24576, 4096, 2048, 256, None, BF, (ONE, 128, 1, 1)), (8192, 4096, 4096, 1, None, F32, (ONE, 128, 1, 1)),
    (8192, 4096, 4096, 1, "swiglu", F32, (ONE, 64, 1, 1)), (715, 232, 5928, 1, None, F32, (ONE, 32, 1, 1)),
    # long ones
    (16384, 4096, 2048, 1, None, BF, (PAIR, 256, 1, 1)), (4096, 2048, 1024, 1, None, BF, (PAIR, 256, 1, 1)),
    (32768, 2880, 2880, 32, None, BF, (PAIR, 256, 1, 1)),
    # with swiglu, whose tiles of 128 rows cost more loads: in pairs down to some 250 rows a group
    (32768, 5760, 2880, 32, "swiglu", BF, (PAIR, 256, 1, 1)), (32768, 4096, 2048, 64, "swiglu", BF, (PAIR, 256, 1, 1)),
    (8192, 4096, 2048, 8, "swiglu", BF, (PAIR, 256, 1, 1)), (24576, 4096, 2048, 256, "swiglu", BF, (ONE, 128, 1, 1))])
def test_sizes_take_their_kernel(M, N, K, G, act, out, plan):
    # (at most 32 clusters of four: as many as GPCs of 16 SMs and more hold on any GPU)
    assert _plan(M, N, K, G, G > 1, act, out) == (0, plan)


# ---------------------------------------------------------------- every kernel's results

def _forms(act, out):
    """Every kernel that an output type and activation have."""
    gated = act == "swiglu"
    forms = [(ONE, 32, 1), (ONE, 64 if gated and out == F32 else 128, 1)]
    if out == BF:
        forms.append((PAIR, 256, 1))
    return forms + [(SPLIT, tn, s) for tn in (16, 32, 64, 128) for s in (2, 4, 8) if not (gated and tn > 64)]


def _check_form(plan, X, W, lens, b, r, act, out, grouped=True):
    """One kernel with Z and the residual in place, then bare, against the oracle; rows behind stay as they were."""
    M, width = X.shape[0], W.shape[1] // 2 if act == "swiglu" else W.shape[1]
    x, w, bd = X.to(DEV), W.to(DEV), None if b is None else b.to(DEV)
    gl = torch.from_numpy(lens).to(DEV) if grouped else None
    buf = torch.full((M + 5, width), 7.0, dtype=out, device=DEV)
    buf[:M] = r.to(DEV)
    zbuf = torch.full((M + 5, W.shape[1]), 7.0, dtype=BF, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    st = _run(plan, x, w, gl, buf[:M], bd, buf[:M], act, zbuf[:M], err)
    if st == INVALID:
        return False
    assert st == 0 and pgg.read_error(err) == 0, plan
    assert (buf[M:] == 7).all() and (zbuf[M:] == 7).all(), plan
    tl._check(buf[:M], zbuf[:M], X, W, lens, b, r, act, tl.FORMS[act])
    Y = torch.full((M, width), 7.0, dtype=out, device=DEV)
    assert _run(plan, x, w, gl, Y, None, None, act, None, err) == 0 and pgg.read_error(err) == 0
    tl._check(Y, None, X, W, lens, None, None, act, tl.FORMS[act])
    again = torch.zeros_like(Y)
    assert _run(plan, x, w, gl, again, None, None, act, None, err) == 0
    assert torch.equal(Y, again), plan
    return True


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("N,K,lens", [
    (272, 1096, [130, 0, 53]),        # every kernel has it; column tiles that end inside a kernel's
    (16, 520, [1]), (1040, 72, [70, 0, 260])])
def test_every_kernel(N, K, lens, act, out):
    lens = np.array(lens, dtype=np.int32)
    X, W, b, r = tl._inputs(int(lens.sum()), N, K, lens, N + K, act=act, out=out)
    ran = [p for p in _forms(act, out) if _check_form(p, X, W, lens, b, r, act, out)]
    # (a kernel that cuts K needs two k-blocks a CTA; for fp32 results four times its accumulators at most)
    nkb = -(-K // 64)
    H = 2 if act == "swiglu" else 1
    assert ran == [p for p in _forms(act, out) if p[0] != SPLIT or (
        nkb >= 2 * p[2] and (out == BF or -(-nkb // p[2]) <= 4 * min(-(-nkb // p[2]), 256 // (H * p[1]))))]


@pytest.mark.gpu
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("N,K,lens", [
    (336, 328, [300, 0, 1, 257, 16, 31]),    # ragged rows over the two CTAs, a CTA without columns
    (528, 64, [513]), (176, 456, [15, 0, 0, 48, 255, 256])])
def test_pairs_of_ctas(N, K, lens, act):
    lens = np.array(lens, dtype=np.int32)
    X, W, b, r = tl._inputs(int(lens.sum()), N, K, lens, N + K, act=act)
    assert _check_form((PAIR, 256, 1), X, W, lens, b, r, act, BF, grouped=len(lens) > 1)
    if len(lens) == 1:
        assert _check_form((PAIR, 256, 1), X, W, lens, b, r, act, BF)


@pytest.mark.gpu
@pytest.mark.parametrize("act,M,N,K", [(None, 5130, 1040, 1032), ("swiglu", 5130, 1040, 264)])
def test_pairs_walk_several_tiles(act, M, N, K):
    # more tiles than pairs: both accumulators in turn, the residual's rows fetched ahead
    lens = np.array([M - 1290, 1290], dtype=np.int32)
    assert sum(-(-lens // 256)) * 5 > 76
    X, W, b, r = tl._inputs(M, N, K, lens, 3, act=act)
    x, w = X.to(DEV), W.to(DEV)
    gl = torch.from_numpy(lens).to(DEV)
    outs = {}
    for plan in ((PAIR, 256, 1), (ONE, 128, 1)):
        Y = torch.zeros(M, N // 2 if act == "swiglu" else N, dtype=BF, device=DEV)
        Z = torch.zeros(M, N, dtype=BF, device=DEV)
        for _ in range(3):
            assert _run(plan, x, w, gl, Y, b.to(DEV), r.to(DEV), act, Z) == 0
        outs[plan] = Y, Z
    tl._check(*outs[PAIR, 256, 1], X, W, lens, b, r, act, tl.FORMS[act])
    # the kernels add up K in the same steps: the results are the same but for the order within an MMA
    for u, v in zip(*outs.values()):
        util.assert_close(u, util.f64(v), "pair against one", rel=2 ** -7, abs_rms=2 ** -12)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("act,M,N,K,tn,splits", [(None, 45, 2568, 1032, 16, 4), ("swiglu", 70, 3088, 1032, 32, 4),
                                                 ("silu", 61, 2440, 2504, 32, 8)])
def test_clusters_with_two_ctas_an_sm(act, M, N, K, tn, splits, out):
    lens = np.array([M], dtype=np.int32)
    X, W, b, r = tl._inputs(M, N, K, lens, 3, act=act, out=out)
    width = N // 2 if act == "swiglu" else N
    assert -(-M // tn) * -(-width // 128) * splits > 152   # CTAs of the launch: more than SMs
    assert _check_form((SPLIT, tn, splits), X, W, lens, b, r, act, out, grouped=False)


@pytest.mark.gpu
def test_the_call_takes_the_planned_kernel():
    # the public call at sizes of each kernel gives the bits of the kernel that the plan names
    for M, N, K, G, act, out in ((3219, 192, 6704, 1, None, BF), (146, 2784, 8024, 1, "swiglu", BF), (5, 512, 1024, 1, "silu", F32),
                                 (4096, 2048, 1024, 1, "gelu", BF), (900, 512, 512, 3, "swiglu", F32)):
        lens = tl._split(np.random.default_rng(M), M, G)
        X, W, b, r = (t.to(DEV) for t in tl._inputs(M, N, K, lens, 1, act=act, out=out))
        gl = None if G == 1 else torch.from_numpy(lens).to(DEV)
        st, plan = _plan(M, N, K, G, G > 1, act, out)
        Y = torch.empty_like(r)
        assert st == 0 and _run(plan[:3], X, W, gl, Y, b, r, act) == 0
        got, _ = pgg.grouped_linear(X, W, gl, bias=b, residual=r, act=act, out_dtype=out, **tl.FORMS[act])
        assert torch.equal(Y, got), plan


# ---------------------------------------------------------------- overlap, and loads that stop

@pytest.mark.gpu
def test_kernels_of_every_form_on_four_streams_at_once():
    work = []
    for i, (plan, M, N, K, G, act, out) in enumerate([
            ((PAIR, 256, 1), 2500, 528, 520, 2, "swiglu", BF), ((SPLIT, 16, 4), 45, 2568, 1032, 1, None, F32),
            ((SPLIT, 32, 4), 70, 3088, 1032, 1, "swiglu", F32), ((SPLIT, 64, 4), 300, 640, 2056, 2, "swiglu", BF),
            ((PAIR, 256, 1), 3000, 768, 520, 1, "gelu", BF), ((SPLIT, 128, 2), 700, 256, 2056, 1, "silu", BF),
            ((SPLIT, 32, 8), 61, 2440, 2504, 1, None, BF), ((ONE, 128, 1), 1500, 512, 520, 3, "silu", F32)]):
        lens = tl._split(np.random.default_rng(i), M, G)
        X, W, b, r = (t.to(DEV) for t in tl._inputs(M, N, K, lens, i, act=act, out=out))
        a = (plan, X, W, torch.from_numpy(lens).to(DEV))
        ref = torch.empty_like(r)
        assert _run(*a, ref, b, r, act) == 0
        work.append((a, b, r, act, ref))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for n in range(40):
        for j, s in enumerate(streams):
            a, b, r, act, ref = work[(n + 3 * j) % len(work)]
            with torch.cuda.stream(s):
                Y = torch.empty_like(ref)
                assert _run(*a, Y, b, r, act) == 0
                got.append((Y, ref))
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in got)


@pytest.mark.gpu
@pytest.mark.parametrize("stall_at", [0, 3, 9])
@pytest.mark.parametrize("plan,M,N,act", [
    ((PAIR, 256, 1), 600, 512, None), ((PAIR, 256, 1), 600, 512, "swiglu"), ((SPLIT, 64, 2), 100, 256, "swiglu"),
    ((SPLIT, 128, 4), 200, 256, None), ((SPLIT, 32, 4), 64, 2560, None), ((ONE, 128, 1), 600, 512, "swiglu")])
def test_loads_that_stop(plan, M, N, act, stall_at):
    """The kernel gives up within its limit, says so, and the next calls are right."""
    K = 1024
    X, W = torch.ones(M, K, dtype=BF, device=DEV), torch.ones(1, N, K, dtype=BF, device=DEV)
    Y = torch.zeros(M, N // 2 if act else N, dtype=BF, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    form = {"alpha": 0.0, "limit": 2.0} if act else {"alpha": 1.0}
    assert _run(plan, X, W, None, Y, act=act, err=err, stall_at=stall_at, wait_ns=2_000_000, **form) == 0
    assert pgg.read_error(err) == 17
    err.zero_()
    assert _run(plan, X, W, None, Y, act=act, err=err, **form) == 0
    assert pgg.read_error(err) == 0 and (Y == (2.0 if act else K)).all()   # 2 sigmoid(0) 2
