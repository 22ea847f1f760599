"""MoeBlock routes by fp32 logits: experts whose logits differ by less than a bf16 step are told apart, and an output is
off by its own roundings, not by its logits'.

A logit is a sum of H = 256 products in fp32, one accumulator of the tensor core: (H / 16 + 16) 2^-23 of the magnitudes."""
import numpy as np
import pytest
import torch

import test_block_parts as parts
from test_block_parts import DEV, H, _block, _t
import util

pgg = pytest.importorskip("precision_grouped_gemm_gb300")
pytestmark = pytest.mark.gpu


def _logits(b, y):
    y, g = util.f64(y), util.f64(b.gate)
    return y @ g.T, (H / 16 + 16) * 2.0 ** -23 * (np.abs(y) @ np.abs(g).T)


@pytest.mark.parametrize("T", [1, 40, 700])
def test_logits_are_fp32(T):
    rng, b = _block(31)
    x, res = _t(rng, T, H), _t(rng, T, H)
    _, _, saved = b.forward(x, res, rng=torch.tensor([1, 2], device=DEV))
    ref, bound = _logits(b, saved[1])
    assert saved[3].dtype == torch.float32
    assert (np.abs(saved[3].double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.parametrize("T", [4, 300])
def test_experts_closer_than_a_bf16_step_are_told_apart(T):
    # every second expert's gate is its neighbour's but for one small number: logits some 2^-10 apart
    rng, b = _block(32, biased=False, shared=False, join=False)
    b.k = 1
    gate = b.gate.clone()
    gate[:, 0] = gate[:, 0].abs().clamp(0.0625, 0.12)   # (the small number is representable beside it)
    gate[1::2] = gate[::2]
    gate[1::2, 0] += 2.0 ** -10
    b.gate = gate
    x, res = _t(rng, T, H), _t(rng, T, H)
    out, _, saved = b.forward(x, res)
    ref, bound = _logits(b, saved[1])
    best = np.sort(ref, axis=1)
    sure = best[:, -1] - best[:, -2] > 2 * bound.max(axis=1)
    near = (best[:, -1] - best[:, -2]) / np.abs(best[:, -1]) < 2.0 ** -9
    assert (sure & near).sum() >= 0.5 * T
    ids = saved[4].cpu().numpy()[:, 0]
    assert np.array_equal(ids[sure], ref.argmax(axis=1)[sure])
    decoded = b.decode(x[:4], res[:4])[0]
    assert not torch.isnan(decoded).any()


@pytest.mark.parametrize("seed", range(8))
def test_block_with_all_parts_whatever_the_gate(seed):
    # the composition's own test with the gates of eight seeds (its inputs are not seeded)
    torch.cuda.manual_seed(seed)
    parts.test_block_with_all_parts("row")
