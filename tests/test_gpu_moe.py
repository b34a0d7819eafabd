"""GPU tests of the mixture-of-experts token movement: the sort and the copies
exactly, the sums against 64 bits.

Tolerances.  combine: fp32 sums of at most 65 terms, then one rounding to bf16
(2^-8 of the value): |err| <= 2^-8 |ref| + 66 * 2^-23 * sum |terms|.
dweights: fp32 dot product of h terms, at most ceil(h / 64) terms in a chain per lane
and 16 more in the tree: |err| <= (h / 64 + 18) 2^-24 sum |terms|."""
import numpy as np
import pytest
import torch

import oracle
from _block_ref import f64, sort
from _helpers import dev_scalar, nv, require_library, syn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def _ids(tokens, topk, experts, seed, dtype=torch.int32, drop=0.1):
    g = torch.Generator().manual_seed(seed)
    skew = torch.randn(experts, generator=g) * 2
    ids = torch.multinomial(torch.softmax(skew, 0).expand(max(tokens, 1), experts), topk, generator=g, replacement=topk > experts)
    ids = ids[:tokens]
    out = torch.rand(ids.shape, generator=g)
    ids = torch.where(out < drop / 2, -1, torch.where(out < drop, experts + 3, ids))
    return ids.to(dtype)


def _bf16(shape, seed):
    return syn.bf16_normal(shape, 1.0, seed).cuda()


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 8, 64), (5, 2, 3), (333, 3, 40), (1024, 1, 7),
                                                 (4000, 6, 257), (700, 2, 1024), (60000, 4, 128)])
def test_sort(tokens, topk, experts, dtype):
    ids = _ids(tokens, topk, experts, tokens + experts, dtype)
    offsets, counts, dest = nv.moe_sort(ids.cuda(), experts)
    o, c, d = sort(ids.numpy(), experts)
    assert np.array_equal(offsets.cpu().numpy(), o)
    assert np.array_equal(counts.cpu().numpy(), c)
    assert np.array_equal(dest.cpu().numpy(), d)
    assert o[-1] <= nv.nvfp4_moe_rows(tokens, topk, experts)


def test_sort_extremes():
    """Every assignment dropped; every one to the last expert; ids of the type's extremes; no tokens."""
    for ids in (torch.full((300, 4), -1), torch.full((1500, 2), 8), torch.tensor([[-2 ** 62, 2 ** 62, 3, 2 ** 32 + 1]])):
        offsets, counts, dest = nv.moe_sort(ids.cuda(), 9)
        o, c, d = sort(ids.numpy(), 9)
        assert np.array_equal(offsets.cpu().numpy(), o) and np.array_equal(dest.cpu().numpy(), d)
        assert np.array_equal(counts.cpu().numpy(), c)
    offsets, counts, dest = nv.moe_sort(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 5)
    assert not offsets.any() and not counts.any() and dest.shape == (0, 4)


def _sorted(tokens, topk, experts, seed, drop=0.1):
    ids = _ids(tokens, topk, experts, seed, drop=drop).cuda()
    return nv.moe_sort(ids, experts)


SHAPES = [(1, 1, 1, 8), (1, 8, 16, 2048), (77, 3, 5, 20), (300, 2, 40, 4104), (513, 6, 8, 264), (40, 64, 16, 96)]


@pytest.mark.parametrize("tokens,topk,experts,h", SHAPES)
def test_dispatch(tokens, topk, experts, h):
    offsets, counts, dest = _sorted(tokens, topk, experts, h)
    rows = nv.nvfp4_moe_rows(tokens, topk, experts)
    ld = (h + 7) // 8 * 8 + 8
    x = _bf16((tokens, ld), h)[:, :h]
    out = torch.full((rows, ld), -3.0, dtype=torch.bfloat16, device="cuda")
    nv.moe_dispatch(x, dest, offsets, counts, out=out[:, :h])
    torch.cuda.synchronize()
    want = torch.full((rows, ld), -3.0, dtype=torch.bfloat16)
    want[:int(offsets[-1]), :h] = 0
    d = dest.cpu().long()
    for t, k in zip(*np.nonzero(d.numpy() >= 0)):
        want[d[t, k], :h] = x[t].cpu()
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("tokens,topk,experts,h", SHAPES)
def test_dispatch_quant(tokens, topk, experts, h):
    """Codes and scales of every row are the oracle's; padding rows are not written."""
    offsets, counts, dest = _sorted(tokens, topk, experts, h)
    rows = nv.nvfp4_moe_rows(tokens, topk, experts)
    ld = (h + 7) // 8 * 8
    x = _bf16((tokens, ld), h)[:, :h]
    gs = syn.global_scale(x)
    x_fp4 = torch.full((rows, nv.padded_k(h) // 2), 0xA5, dtype=torch.uint8, device="cuda")
    x_sf = torch.full((nv.nvfp4_scale_bytes(rows, h),), 0xA5, dtype=torch.uint8, device="cuda")
    nv.nvfp4_moe_dispatch_quant(x, ld, dev_scalar(gs), dest, tokens, topk, rows, h, x_fp4, x_sf)
    torch.cuda.synchronize()
    q, sf = oracle.quantize(syn.bf16_bits(x), gs)
    cols = nv.scale_shape(rows, h)[1]
    got_q, got_sf = x_fp4.cpu().numpy(), oracle.unswizzle(x_sf.cpu().numpy(), rows, cols)
    want_q, want_sf = np.full_like(got_q, 0xA5), np.full_like(got_sf, 0xA5)
    d = dest.cpu().numpy()
    for t, k in zip(*np.nonzero(d >= 0)):
        want_q[d[t, k]] = q[t]
        want_sf[d[t, k]] = 0
        want_sf[d[t, k], :sf.shape[1]] = sf[t]
    assert np.array_equal(got_q, want_q) and np.array_equal(got_sf, want_sf)


def _terms(y, w, dest, res):
    d = dest.cpu().numpy()
    rows = np.where(d[..., None] >= 0, f64(y)[np.maximum(d, 0)], 0.0)
    terms = rows * (f64(w)[..., None] if w is not None else 1.0)
    return np.concatenate([terms, f64(res)[:, None]], 1) if res is not None else terms


@pytest.mark.parametrize("weights,residual", [(True, False), (True, True), (False, False)])
@pytest.mark.parametrize("tokens,topk,experts,h", SHAPES)
def test_combine(tokens, topk, experts, h, weights, residual):
    offsets, counts, dest = _sorted(tokens, topk, experts, h)
    rows = nv.nvfp4_moe_rows(tokens, topk, experts)
    ld = (h + 7) // 8 * 8 + 16
    y = _bf16((rows, ld), h + 1)[:, :h]
    y[int(offsets[-1]):] = float("nan")                     # rows no assignment has
    w = torch.rand((tokens, topk), device="cuda") if weights else None
    if weights:
        w[dest < 0] = float("nan")                          # weights of dropped assignments
    res = _bf16((tokens, ld), h + 2)[:, :h] if residual else None
    out = torch.full((tokens, ld), -3.0, dtype=torch.bfloat16, device="cuda")
    nv.moe_combine(y, dest, w, res, out=out[:, :h])
    torch.cuda.synchronize()
    assert (out[:, h:] == -3.0).all()
    terms = _terms(y, None if w is None else torch.nan_to_num(w), dest, res)
    ref = terms.sum(1)
    err = np.abs(f64(out[:, :h]) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 66 * 2.0 ** -23 * np.abs(terms).sum(1)).all()


def test_combine_of_dropped_tokens_is_the_residual():
    dest = torch.full((6, 3), -1, dtype=torch.int32, device="cuda")
    y = torch.full((128, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    res = _bf16((6, 64), 1)
    assert torch.equal(nv.moe_combine(y, dest, residual=res), res)
    assert not nv.moe_combine(y, dest).any()


@pytest.mark.parametrize("tokens,topk,experts,h", SHAPES)
def test_combine_backward(tokens, topk, experts, h):
    offsets, counts, dest = _sorted(tokens, topk, experts, h)
    rows = nv.nvfp4_moe_rows(tokens, topk, experts)
    ld = (h + 7) // 8 * 8 + 8
    y, dout = _bf16((rows, ld), h + 1)[:, :h], _bf16((tokens, ld), h + 2)[:, :h]
    w = torch.rand((tokens, topk), device="cuda")
    w[dest < 0] = float("nan")
    dy = torch.full((rows, ld), -3.0, dtype=torch.bfloat16, device="cuda")
    _, dw = nv.moe_combine_backward(dout, y, w, dest, offsets, counts, dy=dy[:, :h])
    torch.cuda.synchronize()
    want = torch.full((rows, ld), -3.0, dtype=torch.bfloat16)
    want[:int(offsets[-1]), :h] = 0
    d = dest.cpu()
    for t, k in zip(*np.nonzero(d.numpy() >= 0)):
        want[int(d[t, k]), :h] = (dout[t].cpu().float() * w[t, k].cpu()).to(torch.bfloat16)
    assert torch.equal(dy.cpu(), want)
    terms = f64(dout)[:, None] * np.where(d.numpy()[..., None] >= 0, f64(y)[np.maximum(d.numpy(), 0)], 0.0)
    err = np.abs(f64(dw) - terms.sum(-1))
    assert (err <= (h / 64 + 18) * 2.0 ** -24 * np.abs(terms).sum(-1)).all()
    assert not dw[dest < 0].any()


def test_gradients_against_differences():
    """combine is linear in y and in the weights: a difference of two forward calls is the
    gradient times the step.  Inputs are small integers and steps powers of two, so every
    product, sum and output is exact and the comparison is too."""
    tokens, topk, experts, h = 9, 3, 4, 40
    offsets, counts, dest = _sorted(tokens, topk, experts, 5, drop=0.3)
    rows = nv.nvfp4_moe_rows(tokens, topk, experts)
    g = torch.Generator().manual_seed(7)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    y, dout = ints(rows, h), ints(tokens, h)
    w = torch.randint(0, 4, (tokens, topk), generator=g).float().cuda()
    dy, dw = nv.moe_combine_backward(dout, y, w, dest, offsets, counts)
    loss = lambda yy, ww: (f64(nv.moe_combine(yy, dest, ww)) * f64(dout)).sum()  # noqa: E731
    for t, k in [(0, 0), (3, 1), (8, 2), (5, 0)]:
        step = torch.zeros_like(w)
        step[t, k] = 1.0
        assert (loss(y, w + step) - loss(y, w - step)) / 2 == float(dw[t, k])
        r = int(dest[t, k])
        if r >= 0:
            for c in (0, 17, 39):
                step = torch.zeros_like(y)
                step[r, c] = 1.0
                assert (loss(y + step, w) - loss(y - step, w)) / 2 == float(dy[r, c])
    # dispatch's gradient is combine without weights
    x, drows = ints(tokens, h), ints(rows, h)
    drows[int(offsets[-1]):] = 0
    base = torch.zeros((rows, h), dtype=torch.bfloat16, device="cuda")
    fwd = lambda xx: (f64(nv.moe_dispatch(xx, dest, offsets, counts, out=base.clone())) * f64(drows)).sum()  # noqa: E731
    dx = nv.moe_combine(drows, dest)
    for t, c in [(0, 0), (4, 21), (8, 39)]:
        step = torch.zeros_like(x)
        step[t, c] = 1.0
        assert (fwd(x + step) - fwd(x - step)) / 2 == float(dx[t, c])


def test_rows_past_the_buffer_are_dropped():
    """A dest that does not belong to the buffer is not followed out of it."""
    dest = torch.tensor([[0, 500]], dtype=torch.int32, device="cuda")
    y = _bf16((128, 64), 3)
    assert torch.equal(nv.moe_combine(y, dest), y[:1])


def test_results_repeat_on_another_stream():
    offsets, counts, dest = _sorted(2000, 8, 64, 9)
    y, dout = _bf16((nv.nvfp4_moe_rows(2000, 8, 64), 520), 1), _bf16((2000, 520), 2)
    w = torch.rand((2000, 8), device="cuda")
    dy, dw = torch.zeros_like(y), None
    _, dw = nv.moe_combine_backward(dout, y, w, dest, offsets, counts, dy=dy)
    out = nv.moe_combine(y, dest, w, dout)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        dy2 = torch.zeros_like(y)
        _, dw2 = nv.moe_combine_backward(dout, y, w, dest, offsets, counts, dy=dy2)
        out2 = nv.moe_combine(y, dest, w, dout)
    s.synchronize()
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2) and torch.equal(out, out2)
