"""GPU tests of the choice of experts where fp32 keys cannot tell: against keys in 64 bits, id by id."""
import numpy as np
import pytest
import torch

import _train_ref as ref
from _helpers import require_library
from test_gpu_route import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def biased(l, target, score):
    """(logits [1, e], bias) on the GPU: the bias that brings each key to its target, rounded to fp32."""
    s = ref.scores(l[None].astype(np.float64), score)[0]
    return torch.from_numpy(l[None]).cuda(), torch.from_numpy((target - s).astype(np.float32)).cuda()


def rounding_one_way(e, count):
    """Logits -c whose exponentials lie just off half a step of 1, so that a sequential fp32 sum of 1 and a lane's
    others is off by its length in half steps: (c, error of the sum) of the `count` largest errors each way."""
    rng = np.random.default_rng(e)
    terms = (1 << int(np.ceil(np.log2(e / 32)))) - 1
    c = rng.uniform(6.5, 9.0, 20000).astype(np.float32)
    x = np.exp(-c.astype(np.float64)).astype(np.float32)
    part = np.ones_like(x)
    for _ in range(terms):
        part += x
    off = part - (1.0 + terms * x.astype(np.float64))
    order = np.argsort(off)
    return [(c[i], off[i]) for i in np.concatenate([order[:count], order[-count:]])]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,topk", [(64, 2), (256, 2), (256, 8), (1000, 5), (1024, 31)])
def test_left_out_expert_near_a_pick_that_is_not_the_last(e, topk, score):
    """Two picks whose keys share their upper bits, so that the expert's number puts the higher one last; two
    left-out experts within two steps of the lower one, on the other side of a change of those bits."""
    rng = np.random.default_rng(e + topk)
    step, bucket = 2.0 ** -24, 32 * (1 << max(0, int(np.ceil(np.log2(e / 32)))))
    for _ in range(300):
        target = rng.uniform(-0.5, 0.5, e)
        target[:topk - 2] = 0.85 + 0.1 * rng.random(topk - 2)
        target[topk - 2] = 0.75 + step * bucket * rng.uniform(0.3, 0.8)
        target[topk - 1:topk + 2] = 0.75 + step * rng.uniform(-0.9, 0.9, 3)
        l, bias = biased(rng.standard_normal(e).astype(np.float32), rng.permutation(target), score)
        check(l, topk, score, bias)


@pytest.mark.parametrize("e,topk", [(256, 1), (1024, 1), (1024, 4)])
def test_left_out_expert_with_a_large_score(e, topk):
    """The second left-out expert has nearly all of the softmax, and with it all of its error; the pick and the
    first one left out have little."""
    rng = np.random.default_rng(e + topk)
    for c0, off in rounding_one_way(e, 12):
        l = np.full(e, -c0, np.float32)
        l[0] = 0.0
        for gap in (1.0, 2.0, 4.0):                          # (the fp32 key of expert 0 is off by -off of its score)
            target = rng.uniform(-1.0, -0.5, e)
            target[e - topk:e - 1] = 0.5 + 0.1 * rng.random(topk - 1)
            target[e - 1], target[0] = 32 * 2.0 ** -24, (32 + gap) * 2.0 ** -24
            target[1] = 24 * 2.0 ** -24
            logits, bias = biased(l, target, "softmax")
            check(logits, topk, "softmax", bias)


@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (2, 1)])
@pytest.mark.parametrize("e", [64, 256, 512, 1024])
def test_sums_of_exponentials_that_round_one_way(e, groups, topk_groups):
    """One score near 1 and others equal, their exponential just off half a step of the sum: the fp32
    sum of a lane's exponentials is off by its length in half steps, and all scores with it."""
    for c0, _ in rounding_one_way(e, 12):
        l = np.full(e, -c0, np.float32)
        l[0] = 0.0
        for delta in (-2.0, -1.0, -0.5, 0.5, 1.0, 2.0):
            target = np.full(e, -1.0)
            target[0], target[e - 1] = 0.0, delta * 2.0 ** -24
            logits, bias = biased(l, target, "softmax")
            check(logits, 1, "softmax", bias, groups=groups, topk_groups=topk_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [16.0, 1024.0, 2.0 ** 20])
@pytest.mark.parametrize("e,groups", [(64, 8), (96, 3), (256, 8)])
def test_biases_that_cancel_in_a_group(e, groups, size, score):
    """A group's two highest keys are a large bias and its negative: the sum is far smaller than their roundings."""
    g = torch.Generator(device="cuda").manual_seed(e)
    l = torch.randn(400, e, device="cuda", generator=g) * 2.0 ** -13 * size / 1024
    bias = torch.full((groups, e // groups), -float("inf"), device="cuda")
    bias[:, 1], bias[:, 3] = size, -size
    check(l, 4, score, bias.reshape(-1), groups=groups, group_top=2, topk_groups=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [32, 96])
def test_groups_of_the_lowest_bias_stand_before_empty_ones(e, score):
    """Masks of the type's lowest value: two such keys add up to -inf in fp32, and yet they are keys."""
    l = torch.randn(6, 4, e // 4, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    bias = torch.zeros(4, e // 4, device="cuda")
    l[:, [1, 3]] = -float("inf")
    l[4, 0] = -float("inf")
    l[5, 0, 1:] = -float("inf")
    bias[2] = torch.finfo(torch.float32).min
    check(l.reshape(6, e), e // 4 + 4, score, bias.reshape(-1), groups=4, group_top=2, topk_groups=2)
    bias[2, 0] = -torch.finfo(torch.float32).min
    check(l.reshape(6, e), e // 4 + 4, score, bias.reshape(-1), groups=4, group_top=2, topk_groups=2)
