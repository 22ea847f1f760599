"""What MoeBlock.forward hands to its backward pass: on its own whatever the caller does with the arguments."""
import pytest
import torch

from test_block_parts import DEV, H, _block, _t

pytestmark = pytest.mark.gpu


def _grads(step):
    """The gradients of a block with dropout whose generator state is stepped on by `step` between the passes."""
    rng, b = _block(17)
    x, res, dout, dh = (_t(rng, 40, H) for _ in range(4))
    state = torch.tensor([5, 70], device=DEV)
    out, h, saved = b.forward(x, res, rng=state)
    step(state)
    return out, h, b.backward(dout, dh, saved)


def test_backward_has_the_mask_of_its_forward():
    out, h, ref = _grads(lambda s: None)
    for step in (lambda s: s[1].add_(1), lambda s: s.zero_(), lambda s: s.copy_(torch.tensor([-1, 2 ** 40]))):
        out2, h2, got = _grads(step)
        assert torch.equal(out, out2) and torch.equal(h, h2)
        for name in ref:
            assert torch.equal(ref[name], got[name]), name


def test_layers_share_a_state_that_is_stepped_between_them():
    rng, b = _block(18)
    x, res, dout, dh = (_t(rng, 24, H) for _ in range(4))
    state = torch.tensor([5, 70], device=DEV)
    alone = []
    for i in range(3):
        saved = b.forward(x, res, rng=torch.tensor([5, 70 + i], device=DEV))[2]
        alone.append(b.backward(dout, dh, saved))
    saved = []
    for _ in range(3):
        saved.append(b.forward(x, res, rng=state)[2])
        state[1] += 1
    for ref, s in zip(alone[::-1], saved[::-1]):
        got = b.backward(dout, dh, s)
        assert all(torch.equal(ref[n], got[n]) for n in ref)
    assert not torch.equal(alone[0]["dx"], alone[1]["dx"])


def test_both_passes_in_a_graph_that_steps_the_state_between_them():
    rng, b = _block(19)
    x, res, dout, dh = (_t(rng, 24, H) for _ in range(4))
    state = torch.tensor([5, 70], device=DEV)
    b.backward(dout, dh, b.forward(x, res, rng=state)[2])   # (what is made once is made)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, h, saved = b.forward(x, res, rng=state)
        state[1] += 1
        grads = b.backward(dout, dh, saved)
    for i in range(3):
        state.copy_(torch.tensor([9, 30 + i]))
        g.replay()
        assert state.tolist() == [9, 31 + i]
        o, _, s = b.forward(x, res, rng=torch.tensor([9, 30 + i], device=DEV))
        ref = b.backward(dout, dh, s)
        assert torch.equal(out, o) and all(torch.equal(ref[n], grads[n]) for n in ref)


def test_a_plain_block_keeps_only_what_its_backward_reads():
    rng, b = _block(20, join=False)
    x, res, dout, dh = (_t(rng, 24, H) for _ in range(4))
    ref = b.backward(dout, dh, b.forward(x, res)[2])
    at = x.data_ptr()
    out, h, saved = b.forward(x, res)
    assert all(t is None or t.data_ptr() != at for t in saved)
    x.fill_(float("nan"))   # (as if its memory were another's by now)
    got = b.backward(dout, dh, saved)
    assert all(torch.equal(ref[n], got[n]) for n in ref)
