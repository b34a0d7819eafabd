"""GPU tests of expert routing and its gradient against 64-bit references.

Ids are whole numbers and equal.  Weights: expf is good to 2 ulp (2^-22) and l - max is
rounded to 2^-24 of itself, which for logits within +-32 moves an exponential by 2^-18; a
quotient of such sums stays within 2^-16.  The gradient's terms have the same relative error, so
its error is at most 2^-15 of the sum of their magnitudes, and for bf16 half a step more."""
import numpy as np
import pytest
import torch

import _train_ref as ref
from _helpers import nv, require_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def logits_of(t, e, bf16, seed, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn(t, e, device="cuda", generator=g) * std
    return l.to(torch.bfloat16) if bf16 else l


def check(logits, topk, score="softmax", bias=None, renorm=True, scale=1.0, rel=2.0 ** -16, **groups):
    ids, w = nv.moe_route(logits, topk, score, bias, renormalize=renorm, scale=scale, **groups)
    torch.cuda.synchronize()
    l = logits.double().cpu().numpy()
    want = ref.choose(l, topk, score, None if bias is None else bias.cpu().numpy(), **groups)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:4]
    wref = ref.weights(l, want, score, renorm, scale)
    wgot = w.double().cpu().numpy()
    assert np.all(np.abs(wgot - wref) <= rel * np.abs(wref) + 2.0 ** -126)
    assert np.all(wgot[want < 0] == 0)
    return ids, w


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("t,e,topk", [(1, 1, 1), (1, 8, 2), (5, 33, 8), (130, 60, 6), (64, 128, 8), (67, 160, 3),
                                      (9, 256, 8), (31, 513, 10), (6, 1024, 64), (4, 64, 64)])
def test_plain(t, e, topk, renorm, score, bf16):
    check(logits_of(t, e, bf16, t + e), topk, score, None, renorm, 2.5)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("e,groups,topk_groups,topk", [(256, 8, 4, 8), (64, 8, 1, 8), (160, 5, 2, 6), (32, 32, 7, 7),
                                                       (1024, 32, 3, 20), (6, 2, 1, 3), (96, 3, 3, 4),
                                                       (64, 8, 1, 12), (344, 8, 4, 8), (40, 4, 2, 33)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_and_bias(e, groups, topk_groups, topk, group_top, bias, score, bf16):
    g = torch.Generator(device="cuda").manual_seed(e)
    b = 0.2 * torch.randn(e, device="cuda", generator=g) if bias else None
    check(logits_of(203, e, bf16, e + 1), topk, score, b, groups=groups, group_top=group_top, topk_groups=topk_groups)


@pytest.mark.parametrize("groups,group_top,topk_groups", [(1, 1, 1), (4, 1, 2), (4, 2, 2)])
def test_ties_go_to_the_lower_index(groups, group_top, topk_groups):
    l = torch.tensor([[1.0] * 64, [0.0, -0.0] * 32, [float(i // 8) for i in range(64)], [float(-(i % 3)) for i in range(64)]],
                     device="cuda")
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(64, device="cuda"), torch.full((64,), 3.0, device="cuda")):
            check(l, 9, score, bias, groups=groups, group_top=group_top, topk_groups=topk_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (4, 1), (4, 2)])
@pytest.mark.parametrize("e", [40, 64, 256])
def test_keys_that_fp32_cannot_tell_apart(e, groups, group_top, score):
    """A bias of one target minus the score, rounded to fp32: the keys differ by less than 2^-25."""
    l = logits_of(64, e, False, 3).repeat_interleave(1, 0)
    l[1:] = l[:1]                                            # one row, so that one bias fits all; then its permutations
    g = torch.Generator(device="cuda").manual_seed(4)
    s = torch.from_numpy(ref.scores(l[:1].double().cpu().numpy(), score)[0])
    bias = (0.75 - s).float().cuda()
    key = s + bias.double().cpu()
    assert float(key.max() - key.min()) < 2.0 ** -23
    check(l[:1].contiguous(), 8, score, bias, groups=groups, group_top=group_top, topk_groups=min(2, groups))
    for i in range(8):
        perm = torch.randperm(e, device="cuda", generator=g)
        check(l[:1, perm].contiguous(), 8, score, bias[perm].contiguous(), groups=groups, group_top=group_top,
              topk_groups=min(2, groups))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (4, 1), (4, 2)])
@pytest.mark.parametrize("e,topk", [(24, 3), (64, 8), (256, 8), (1000, 9), (1024, 31), (256, 40)])
@pytest.mark.parametrize("bias", [False, True])
def test_logits_a_few_steps_apart(bias, e, topk, groups, group_top, score):
    """Runs of logits that differ in their last bits, in random order: pairs, triples and many."""
    rng = np.random.default_rng(e + topk)
    base = np.sort(rng.standard_normal(e).astype(np.float32))[::-1].copy()
    rows = []
    for run in (1, 2, 3, e // 2):
        for start in (0, 1, topk - 1, max(topk - 2, 0)):
            l = base.copy()
            n = min(run, e - start)
            l[start:start + n] = l[start] * (1 + np.float32(2.0 ** -23) * rng.integers(0, 9, n).astype(np.float32))
            rows.append(rng.permutation(l))
    b = torch.full((e,), 0.25, device="cuda") if bias else None
    check(torch.from_numpy(np.stack(rows)).cuda(), topk, score, b, groups=groups, group_top=group_top,
          topk_groups=min(3, groups))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_experts_and_rows(renorm, score, bf16):
    inf, nan, low = float("inf"), float("nan"), float(torch.finfo(torch.float32).min)
    l = logits_of(12, 24, bf16, 5)
    l[0] = -inf                                              # nothing left
    l[1] = nan
    l[2, 3:] = -inf                                          # fewer than topk
    l[3, ::2] = nan
    l[4] = low                                               # the type's lowest value is a value
    l[5, 4:] = low
    l[6, 1:] = -inf
    l[7, :20] = -inf
    for groups, group_top, topk_groups in ((1, 1, 1), (4, 1, 2), (4, 2, 2), (24, 2, 5)):
        for bias in (None, torch.linspace(-1, 1, 24, device="cuda")):
            ids, w = check(l, 6, score, bias, renorm, groups=groups, group_top=group_top, topk_groups=topk_groups)
            assert (ids[:2] == -1).all() and (w[:2] == 0).all() and torch.isfinite(w).all()
    bias = torch.zeros(24, device="cuda")
    bias[::3], bias[1] = -inf, nan
    ids, _ = check(l, 6, score, bias, renorm)
    assert not ((ids % 3 == 0) & (ids >= 0)).any() and not (ids == 1).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(score):
    """+inf counts as the largest float; renormalised weights survive any range."""
    inf, big = float("inf"), ref.FLT_MAX
    l = torch.tensor([[inf, 1.0, 2.0, inf, 0, 0], [big, -big, 0, 1, 2, big], [-300.0, -301, -299, -320, -310, -305],
                      [1e4, -1e4, 1e4, 5e3, 0, 1], [-big, -big, -big, -big, -big, -big], [88.8, 103.0, 90, 700, 60, 50]],
                     device="cuda")
    # (l - max of logits of hundreds is exact here or off by 2^-24 of 300: 2^-15.7)
    ids, w = check(l, 3, score, rel=2.0 ** -14)
    assert torch.isfinite(w).all() and torch.allclose(w.sum(1), torch.ones(6, device="cuda"))
    check(l, 3, score, renorm=False, rel=2.0 ** -14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,group_top,topk_groups", [(1, 1, 1), (4, 1, 2), (4, 2, 2), (8, 2, 3)])
def test_infinite_bias(groups, group_top, topk_groups, score):
    """Experts that are always taken beside ones that never are, also as whole groups."""
    l = logits_of(5, 32, False, 15)
    l[1, 8:16] = -float("inf")
    for up, down in (([3], []), ([3, 4, 20], [5]), (range(16), [20]), (range(32), []), ([31], range(24)), (range(8), range(8, 24))):
        bias = torch.zeros(32, device="cuda")
        bias[list(up)], bias[list(down)] = float("inf"), -float("inf")
        check(l, 6, score, bias, groups=groups, group_top=group_top, topk_groups=topk_groups)


def test_strides_and_alignment():
    """Rows of a wider buffer, from an odd element on."""
    for dtype in (torch.float32, torch.bfloat16):
        wide = logits_of(50, 91, dtype == torch.bfloat16, 6)
        view = wide[:, 3:64]
        a, b = nv.moe_route(view, 5), nv.moe_route(view.contiguous(), 5)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        dw = torch.randn(50, 5, device="cuda")
        out = torch.full((50, 91), 7.0, device="cuda").to(dtype)
        nv.nvfp4_moe_route_backward(dw, a[0], view, nv.NVFP4_TYPE_F32 if dtype == torch.float32 else nv.NVFP4_TYPE_BF16,
                                    91, 50, 61, 0, 5, True, 1.0, out[:, 3:], 91)
        torch.cuda.synchronize()
        assert torch.equal(out[:, 3:64], nv.moe_route_backward(dw, a[0], view.contiguous()))
        assert (out[:, :3] == 7).all() and (out[:, 64:] == 7).all()


def test_no_tokens():
    ids, w = nv.moe_route(torch.empty(0, 16, device="cuda"), 4)
    assert ids.shape == w.shape == (0, 4)
    assert nv.moe_route_backward(w, ids, torch.empty(0, 16, device="cuda")).shape == (0, 16)


def check_gradient(logits, ids, dw, score, renorm, scale):
    got = nv.moe_route_backward(dw, ids, logits, score, renorm, scale)
    torch.cuda.synchronize()
    want, mag = ref.route_gradient(dw.double().cpu().numpy(), ids.cpu().numpy().astype(np.int64),
                                   logits.double().cpu().numpy(), score, renorm, scale)
    tol = 2.0 ** -15 * mag + 2.0 ** -120
    if logits.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err / tol).max())
    return got, want


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("t,e,topk", [(1, 1, 1), (1, 8, 2), (5, 33, 8), (130, 60, 6), (67, 160, 3), (31, 513, 10), (6, 1024, 64),
                                      (40, 32, 1), (4, 64, 64)])
def test_gradient(t, e, topk, renorm, score, bf16):
    l = logits_of(t, e, bf16, t + e)
    if t > 4:
        l[2] = -float("inf")
        l[3, 1:] = -float("inf")
        l[4, 0] = float("nan")
    ids, _ = nv.moe_route(l, topk, score, renormalize=renorm, scale=1.5)
    g = torch.Generator(device="cuda").manual_seed(7)
    dw = torch.randn(t, topk, device="cuda", generator=g)
    got, _ = check_gradient(l, ids, dw, score, renorm, 1.5)
    if t > 4:
        assert (got[2] == 0).all() and (got[3, 1:] == 0).all() and got[4, 0] == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(renorm, score):
    """(f(l + h) - f(l - h)) / 2h in 64 bits: off by h^2 of a third derivative below 1, 2^-30, and by rounding 2^-52 / h."""
    l, h, topk = logits_of(3, 20, False, 8), 2.0 ** -15, 4
    ids, _ = nv.moe_route(l, topk, score, renormalize=renorm)
    dw = torch.randn(3, topk, device="cuda")
    got = nv.moe_route_backward(dw, ids, l, score, renorm).double().cpu().numpy()
    base, i, d = l.double().cpu().numpy(), ids.cpu().numpy().astype(np.int64), dw.double().cpu().numpy()
    for c in range(20):
        step = np.zeros((3, 20))
        step[:, c] = h
        f = [(d * ref.weights(base + s * step, i, score, renorm, 1.0)).sum(1) for s in (1, -1)]
        diff = (f[0] - f[1]) / (2 * h)
        assert np.all(np.abs(got[:, c] - diff) <= 2.0 ** -15 * np.abs(d).sum(1)), c


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_given_ids(renorm, score):
    """Ids of another choice: one expert twice, dropped slots, ids out of range."""
    l = logits_of(6, 40, False, 9)
    ids = torch.tensor([[1, 1, 2, 3], [5, 6, 5, 5], [-1, 4, 40, 9], [-1, -1, -1, -1], [0, 39, 38, 39], [7, 8, 9, 1 << 30]],
                       dtype=torch.int32, device="cuda")
    dw = torch.randn(6, 4, device="cuda")
    clipped = torch.where((ids >= 0) & (ids < 40), ids, -1)
    got = nv.moe_route_backward(dw, ids, l, score, renorm)
    _, want = check_gradient(l, clipped, dw, score, renorm, 1.0)
    assert torch.equal(got, nv.moe_route_backward(dw, clipped, l, score, renorm))
    assert (got[3] == 0).all()


def test_one_pick_with_all_the_weight_keeps_its_gradient_exact():
    """Differences of gradients: with weights 1 - 2^-20 and 2^-20 the gradient is theirs, not a rounding."""
    l = torch.tensor([[14.0, 0.0, -5.0]], device="cuda")
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    dw = torch.tensor([[1.0, 1.0 + 2.0 ** -12]], device="cuda")
    got = nv.moe_route_backward(dw, ids, l).double().cpu().numpy()
    want, _ = ref.route_gradient(dw.double().cpu().numpy(), ids.cpu().numpy().astype(np.int64), l.double().cpu().numpy(),
                                 "softmax", True, 1.0)
    assert np.all(np.abs(got - want) <= 2.0 ** -18 * np.abs(want))


def test_captured_and_on_another_stream():
    l = logits_of(300, 64, False, 10)
    bias = torch.randn(64, device="cuda") * 0.1
    ids = torch.zeros(300, 8, dtype=torch.int32, device="cuda")
    w, dl = torch.zeros(300, 8, device="cuda"), torch.zeros(300, 64, device="cuda")
    dw = torch.randn(300, 8, device="cuda")

    def step():
        nv.nvfp4_moe_route(l, 0, 64, bias, 300, 64, 1, 8, 8, 2, 4, True, 2.5, ids, w)
        nv.nvfp4_moe_route_backward(dw, ids, l, 0, 64, 300, 64, 1, 8, True, 2.5, dl, 64)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (11, 12):
        l.copy_(logits_of(300, 64, False, seed))
        graph.replay()
        torch.cuda.synchronize()
        a, b = nv.moe_route(l, 8, "sigmoid", bias, 8, 2, 4, True, 2.5)
        assert torch.equal(a, ids) and torch.equal(b, w)
        assert torch.equal(dl, nv.moe_route_backward(dw, a, l, "sigmoid", True, 2.5))
