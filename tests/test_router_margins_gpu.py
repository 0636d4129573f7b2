"""Groups of experts that nearly tie, among tokens enough that 32 bits order most groups, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import router_helpers as rh
from combine_get_dispatch_amd import ep

pytestmark = pytest.mark.gpu

T = 6000


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def same_choice(logits, r, bias=None):
    """Every token of a batch that fills the chip, and each in a small one, gets the definition's experts."""
    l, b = torch.from_numpy(logits).cuda(), None if bias is None else torch.from_numpy(bias).cuda()
    assert len(l) >= 8 * torch.cuda.get_device_properties(0).multi_processor_count
    want, _ = rh.route(logits, r, bias)
    got = ep.route(l, r, bias=b)[0].cpu().numpy()
    few = torch.cat([ep.route(part.contiguous(), r, bias=b)[0] for part in l.split(1000)]).cpu().numpy()
    for what, idx in (("many", got), ("few", few)):
        bad = np.flatnonzero((idx != want).any(1))
        assert not len(bad), f"{len(bad)} of {what} tokens, {bad[0]}: {idx[bad[0]]}, not {want[bad[0]]}"


@pytest.mark.parametrize("size", [2, 4])
@pytest.mark.parametrize("both", [True, False])
@pytest.mark.parametrize("B", [16.0, 64.0, 1000.0, 1e4])
def test_biases_of_opposite_signs(B, both, size):
    """Of four groups the first is the best and the last the worst; the other two nearly tie: their largest numbers lie near B
    and -B (of one of them, or of both), where 32 bits round them by more than the sums are apart."""
    rng = np.random.default_rng([int(B), int(both), size])
    bias = np.full((4, size), -2 * B, np.float32)
    bias[0, :2], bias[1, :2], bias[2, :2], bias[3, :2] = 2, (B, -B) if both else 0, (B, -B), -2
    x = rng.standard_normal((3 * T, 4, size)).astype(np.float32)
    s = sigmoid(x.astype(np.float64))
    step = float(np.spacing(np.float32(B)))
    apart = rng.choice([-1, 1], 3 * T) * step * np.exp2(rng.uniform(-4, 3, 3 * T))
    last = s[:, 1, 0] + s[:, 1, 1] + apart - s[:, 2, 0]
    last = np.clip(last, 1e-3, 1 - 1e-3)
    x[:, 2, 1] = -np.log(1 / last - 1)
    s = sigmoid(x.astype(np.float64))
    gap = np.abs(s[:, 1, :2].sum(1) - s[:, 2, :2].sum(1))
    # (of a number only 43 leading bits count)
    x = x[(gap > 8 * B * 2.0 ** -42) & (gap < 16 * step)][:T]
    assert len(x) == T
    r = ep.Router(4 * size, 4, score="sigmoid", num_groups=4, topk_groups=2)
    same_choice(x.reshape(T, -1), r, bias.reshape(-1))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("below", [0, 10, 20, 30, 45, 60, 80])
def test_logits_far_below_the_largest(score, below):
    """No bias: of four groups the first has the largest logit and the others' lie `below` under it, where the difference of two
    logits is rounded by more than a score's other roundings; two of them nearly tie."""
    rng = np.random.default_rng([below, int(score == "softmax")])
    of = np.exp if score == "softmax" else sigmoid
    x = (rng.standard_normal((4 * T, 4, 2)) - below / 2).astype(np.float32)
    x[:, 0, 0] = below / 2 + rng.random(4 * T)
    x[:, 3] -= 5
    s = of(x.astype(np.float64))
    first = s[:, 1].sum(1)
    last = first * (1 + rng.choice([-1, 1], 4 * T) * np.exp2(rng.uniform(-24, -16, 4 * T))) - s[:, 2, 0]
    good = (last > 1e-3 * first) & (last < 0.99 if score == "sigmoid" else True)
    x, last = x[good][:T], last[good][:T]
    x[:, 2, 1] = np.log(last) if score == "softmax" else np.log(last) - np.log1p(-last)
    assert len(x) == T
    same_choice(x.reshape(T, 8), ep.Router(8, 4, score=score, num_groups=4, topk_groups=2))


def test_biases_near_the_lowest_number():
    """Groups' sums beyond the lowest 32-bit number: these groups are open, and in order among each other."""
    low = float(np.finfo(np.float32).min)
    bias = np.array([0.5, 0.25, low, low, -1e38, -3e38, -2.9e38, -2.95e38], np.float32)
    logits = np.random.default_rng(1).standard_normal((T, 8)).astype(np.float32)
    r = ep.Router(8, 4, score="sigmoid", num_groups=4, topk_groups=2)
    want, _ = rh.route(logits[:1], r, bias)
    assert sorted(want[0]) == [0, 1, 4, 5]
    same_choice(logits, r, bias)
    same_choice(logits, ep.Router(8, 3, score="sigmoid", num_groups=4, topk_groups=2), np.full(8, low, np.float32))
