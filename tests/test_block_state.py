"""What the few-token layer and the MoE block keep between calls: the workspace after a timeout, and
the quantized weights after an update."""
import copy
import pickle

import numpy as np
import pytest
import torch

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
from precision_grouped_gemm_gb300 import _binding  # noqa: E402
from precision_grouped_gemm_gb300.block import MoeBlock  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FMT = {None: 0, "e4m3": 1, "e2m1": 2}


def _stall(fmt, x, sx, ids, w1, s1, w2, s2, E, ws, err, stall_at=9):
    """A call of the layer whose loads stop, on this workspace: it ends with the timeout code."""
    T, k = ids.shape
    H, I = w2.shape[-2] if w2.dim() == 3 else w2.shape[0] // E, w1.numel() // E // x.shape[1] // 2
    out = torch.zeros(T, H, dtype=BF, device=DEV)
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = _binding.lib().pgg_test_stalled_moe_decode(
        FMT[fmt], p(x), p(sx), p(ids), p(w1), p(s1), p(w2), p(s2), p(out), T, k, H, I, E, stall_at, 2_000_000, p(ws),
        ws.numel(), p(err), torch.cuda.current_stream().cuda_stream)
    assert st == 0


@pytest.mark.parametrize("fmt", [None, "e4m3", "e2m1"])
def test_a_workspace_that_a_timeout_left_is_reported(fmt):
    # sums of the call that gave up are still in the workspace, and the next call cannot tell them from
    # its own: every call on it reports the timeout until it is zeroed
    T, k, E, H, I = 24, 4, 24, 2048, 1024
    g = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF)  # noqa: E731
    ids = torch.from_numpy(np.random.default_rng(3).permuted(np.tile(np.arange(E, dtype=np.int32), (T, 1)), axis=1)
                           [:, :k].copy()).to(DEV)
    x, w1, w2 = rnd(T, H), 0.02 * rnd(E * 2 * I, H), 0.02 * rnd(E * H, I)
    sx = s1 = s2 = None
    if fmt is not None:
        (x, sx), (w1, s1), (w2, s2) = (pgg.mx_quantize_rowwise(x, fmt), pgg.mx_quantize_rowwise_blocked(w1, fmt),
                                       pgg.mx_quantize_rowwise_blocked(w2, fmt))
    ws = pgg.moe_decode_workspace(T, k, H, I, E, fmt)

    def call():
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        if fmt is None:
            out = pgg.moe_decode(x, ids, None, w1.view(E, 2 * I, H), w2.view(E, H, I), ws=ws, err=err)
        else:
            out = pgg.mx_moe_decode(fmt, x, sx, ids, None, w1, s1, w2, s2, ws=ws, err=err)
        return out, pgg.read_error(err)

    good, code = call()
    assert code == 0
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    _stall(fmt, x, sx, ids, w1, s1, w2, s2, E, ws, err)
    assert pgg.read_error(err) == 17
    assert call()[1] == 17 and call()[1] == 17
    ws.zero_()
    out, code = call()
    assert code == 0 and torch.equal(out, good)


def _block(seed, fmt=None, T=24, H=2048, I=1024, E=24, k=4, **kw):
    """A block (the same weights for a seed), and inputs x, residual [T, H]."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s, scale=1.0: (scale * torch.randn(s, generator=g, device=DEV)).to(BF)  # noqa: E731
    b = MoeBlock(1 + rnd(H, scale=0.1), rnd(E, H, scale=0.1), rnd(E, 2 * I, H, scale=H ** -0.5),
                 rnd(E, H, I, scale=I ** -0.5), k, fmt=fmt, **kw)
    return b, rnd(T, H), rnd(T, H)


@pytest.mark.parametrize("fmt", [None, "e4m3", "e2m1"])
@pytest.mark.parametrize("own_word", [True, False])
def test_block_is_ready_again_after_a_timeout(fmt, own_word):
    b, x, res = _block(1, fmt)
    good, _ = b.decode(x, res)
    b.check_decode()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ids = torch.arange(24 * 4, dtype=torch.int32, device=DEV).view(24, 4) % 24
    if fmt is None:
        _stall(fmt, x, None, ids, b.W1, None, b.W2, None, 24, b._ws, b._err if own_word else err)
    else:
        w1, s1, w2, s2 = b._mx
        _stall(fmt, *pgg.mx_quantize_rowwise(x, fmt), ids, w1, s1, w2, s2, 24, b._ws, b._err if own_word else err)
    if own_word:  # the block finds it out by itself
        with pytest.raises(pgg.PggError) as e:
            b.check_decode()
        assert e.value.status == 17
    else:         # the caller, from a word that was given; later calls say so too
        b.decode(x, res, err=err.zero_())
        assert pgg.read_error(err) == 17
        b.prepare_decode()
    for _ in range(2):
        assert torch.equal(b.decode(x, res)[0], good)
    b.check_decode()


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_block_first_decode_inside_a_capture(fmt):
    # what the capture records is not what eager calls use: not before the first replay, nor between replays
    b, x, res = _block(2, fmt)
    good, _ = _block(2, fmt)[0].decode(x, res)  # (another block of the same weights)
    filler = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    del filler  # fresh memory is not zero
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = b.decode(x, res)
    assert torch.equal(b.decode(x, res)[0], good)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, good)
        assert torch.equal(b.decode(x, res)[0], good)
    b.check_decode()
    graph = torch.cuda.CUDAGraph()  # after `prepare_decode` (here: a decode) the capture has the block's own
    with torch.cuda.graph(graph):
        out2, _ = b.decode(x, res)
    for _ in range(2):
        graph.replay()
        assert torch.equal(out2, good) and torch.equal(b.decode(x, res)[0], good)
    b.check_decode()


@pytest.mark.parametrize("fmt", [None, "e4m3", "e2m1"])
def test_block_decode_follows_its_weights(fmt):
    b, x, res = _block(4, fmt, T=9, H=256, I=128, E=8, k=2)
    first, _ = b.decode(x, res)

    def fresh():  # a block that is made of the weights as they are now
        return MoeBlock(b.gamma, b.gate, b.W1.clone(), b.W2.clone(), b.k, fmt=fmt).decode(x, res)[0]

    def check(what):
        out, _ = b.decode(x, res)
        assert torch.equal(out, fresh()), what
        return out

    out = check("no change")
    assert torch.equal(out, first)
    b.W1.mul_(1.5)
    out2 = check("W1 in place")
    assert not torch.equal(out2, out)
    with torch.no_grad():
        b.W2[3:].add_(0.1 * torch.randn_like(b.W2[3:]))
    out3 = check("a part of W2 in place")
    assert not torch.equal(out3, out2)
    for _ in range(3):  # a tensor that takes the place, and often the address, of the one before
        w, b.W1 = b.W1 * 0.5, None
        b.W1 = w
        del w
        check("another W1")
    b.W2 = -b.W2
    check("another W2")
    graph = torch.cuda.CUDAGraph()
    b.W1.neg_()
    with torch.cuda.graph(graph):  # an update that no decode has seen, and then a capture
        out, _ = b.decode(x, res)
    check("before the replay")
    graph.replay()
    assert torch.equal(out, fresh())
    b.W1.data.mul_(2.0)            # torch does not count this: the caller says so
    b.quantize_weights()
    check("told")


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_block_copies_and_blocks_without_bf16_weights(fmt):
    b, x, res = _block(5, fmt, T=5, H=256, I=128, E=8, k=2)
    good, _ = b.decode(x, res)
    for c in (copy.deepcopy(b), pickle.loads(pickle.dumps(b))):
        assert torch.equal(c.decode(x, res)[0], good)
        c.W1.mul_(2.0)
        assert not torch.equal(c.decode(x, res)[0], good)
    assert torch.equal(b.decode(x, res)[0], good)
    if fmt is not None:
        b.W1 = b.W2 = None
        assert torch.equal(b.decode(x, res)[0], good)
        b, x, res = _block(5, fmt, T=5, H=256, I=128, E=8, k=2)
        b.W1 = b.W2 = None  # before the first decode
        assert torch.equal(b.decode(x, res)[0], good)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_block_in_inference_mode(fmt):
    with torch.inference_mode():
        b, x, res = _block(5, fmt, T=5, H=256, I=128, E=8, k=2)
        good, _ = b.decode(x, res)
        assert torch.equal(b.decode(x, res)[0], good)
    ref, _ = _block(5, fmt, T=5, H=256, I=128, E=8, k=2)[0].decode(x, res)
    assert torch.equal(good, ref)
