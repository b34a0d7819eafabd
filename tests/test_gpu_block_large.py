"""Offsets past 2^31 elements and graph capture of the operators around the linear."""
import os
import sys

import pytest
import torch

from _helpers import dev_scalar, nv, require_library, syn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import ffn_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def _spread(rows, stride, make):
    """A [len(rows), cols] tensor's rows written `stride` elements apart, as a strided view."""
    src = make
    full = torch.empty((src.shape[0] - 1) * stride + src.shape[1], dtype=torch.bfloat16, device="cuda")
    view = full.as_strided(src.shape, (stride, 1))
    view.copy_(src)
    return view


def test_norm_rows_past_2_31_elements():
    x = syn.bf16_outlier_channels(3, 4096, 1).cuda()
    r = syn.bf16_outlier_channels(3, 4096, 2).cuda()
    gamma = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    a = nv.add_rmsnorm_quant(x, gamma, 1e-6, residual=r, fmt=nv.NVFP4_FORMAT_MXFP8)
    far = _spread(3, 1 << 30, x)
    b = nv.add_rmsnorm_quant(far, gamma, 1e-6, residual=r, fmt=nv.NVFP4_FORMAT_MXFP8)
    torch.cuda.synchronize()
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_moe_rows_past_2_31_elements():
    tokens, topk, e, h, ld = 40, 2, 3, 64, 1 << 23
    ids = torch.randint(0, e, (tokens, topk), generator=torch.Generator().manual_seed(3)).int().cuda()
    offsets, counts, dest = nv.moe_sort(ids, e)
    rows = nv.nvfp4_moe_rows(tokens, topk, e)
    assert rows * ld > 1 << 31
    x = syn.bf16_normal((tokens, h), 1.0, 4).cuda()
    w = torch.rand((tokens, topk), device="cuda")
    near = torch.zeros((rows, h), dtype=torch.bfloat16, device="cuda")
    far = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").as_strided((rows, h), (ld, 1))
    far.zero_()
    nv.moe_dispatch(x, dest, offsets, counts, out=near)
    nv.moe_dispatch(x, dest, offsets, counts, out=far)
    torch.cuda.synchronize()
    assert torch.equal(near, far)
    assert torch.equal(nv.moe_combine(near, dest, w), nv.moe_combine(far, dest, w))
    g = nv.moe_combine_backward(x, far, w, dest, offsets, counts, dy=far.clone())
    n = nv.moe_combine_backward(x, near, w, dest, offsets, counts, dy=near.clone())
    torch.cuda.synchronize()
    assert torch.equal(g[1], n[1]) and torch.equal(g[0], n[0])


@pytest.mark.parametrize("m", [3, 150])
def test_residual_and_output_rows_past_2_31_elements(m):
    k, n = 256, 136
    stride = (1 << 31) // (m - 1) // 8 * 8 + 64
    x = syn.bf16_outlier_channels(m, k, 5).cuda()
    w = syn.bf16_normal((n, k), 0.05, 6)
    gw = syn.global_scale(w)
    w_fp4, w_sf = nv.prepare_weight(w.cuda(), dev_scalar(gw))
    res = syn.bf16_normal((m, n), 1.0, 7).cuda()
    args = (w_fp4, w_sf, k, n, dev_scalar(20.0), dev_scalar(syn.alpha_of(20.0, gw)))
    a = nv.linear(x, *args, act="silu", residual=res)
    out = torch.empty((m - 1) * stride + n, dtype=torch.bfloat16, device="cuda").as_strided((m, n), (stride, 1))
    nv.linear(x, *args, act="silu", residual=_spread(m, stride, res), out=out)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    assert torch.equal(a, out)


def test_graph_capture_of_both_ffn_blocks():
    """Captured once, replayed on new inputs: equal to the eager calls."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    k, f, e, m = 256, 384, 8, 40
    dense = ffn_block.DenseFFN(1 + rnd(k, std=0.1), rnd(f, k, std=0.05), rnd(f, k, std=0.05), rnd(k, f, std=0.05))
    moe = ffn_block.MoEFFN(rnd(e, k, std=0.1), rnd(e, f, k, std=0.05), rnd(e, f, k, std=0.05), rnd(e, k, f, std=0.05), 2)
    x, r = rnd(m, k), rnd(m, k)
    dense.calibrate(x, r)
    moe.calibrate(x)
    for _ in range(2):
        dense(x, r), moe(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = dense(x, r), moe(x)
    for _ in range(2):
        x.copy_(rnd(m, k))
        r.copy_(rnd(m, k))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, dense(x, r)) and torch.equal(b, moe(x))


@pytest.fixture
def room():
    """room(gb): skips without that much free memory; what a test cached is given back."""
    def need(gb):
        torch.cuda.empty_cache()
        if torch.cuda.mem_get_info()[0] < gb << 30:
            pytest.skip(f"needs {gb} GB of device memory")
    yield need
    torch.cuda.empty_cache()


def test_combine_of_more_than_2_30_tokens(room):
    """topk 1 takes a step of all blocks for (almost) all tokens: the token number plus
    the step passes 2^31.  The expert rows repeat, so the output does."""
    tokens, h, rows = (1 << 30) + 4096 * 3 + 77, 8, 4096
    room(40)
    g = torch.Generator(device="cuda").manual_seed(11)
    y = torch.randn(rows, h, generator=g, device="cuda").bfloat16()
    whole = tokens // rows
    dest = torch.empty(tokens, 1, dtype=torch.int32, device="cuda")
    order = torch.randperm(rows, generator=g, device="cuda").int()
    order[5] = -1                                            # a dropped assignment: zeros
    dest[:whole * rows].view(whole, rows).copy_(order.expand(whole, rows))
    dest[whole * rows:, 0] = order[:tokens - whole * rows]
    out = torch.full((tokens + 8, h), -3.0, dtype=torch.bfloat16, device="cuda")
    nv.moe_combine(y, dest, out=out[:tokens])
    want = y[order.clamp_min(0).long()]
    want[5] = 0
    assert (out[tokens:] == -3.0).all()
    assert torch.equal(out[whole * rows:tokens], want[:tokens - whole * rows])
    full = out[:whole * rows].view(whole, rows * h)
    for i in range(0, whole, 1 << 16):
        assert (full[i:i + (1 << 16)].view(torch.int16) == want.view(1, -1).view(torch.int16)).all(), i


class AlmostTwoToThe31Rows:
    """The largest row count; the rows repeat every 1024, so what is computed row by row does."""
    m, k, period = (1 << 31) - 1024, 8, 1024

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(12)
        self.rows = (torch.randn(self.period, self.k, generator=g, device="cuda") * 3).bfloat16()
        self.x = torch.empty(self.m, self.k, dtype=torch.bfloat16, device="cuda")
        self.x.view(self.m // self.period, -1).copy_(self.rows.view(1, -1).expand(self.m // self.period, -1))

    def check(self, *outputs):
        """(output of x, output of rows) pairs"""
        torch.cuda.synchronize()
        nv.nvfp4_device_error()
        for got, want in outputs:
            got, want = got.view(self.m // self.period, -1), want.view(1, -1)
            for i in range(0, got.shape[0], 1 << 15):
                assert (got[i:i + (1 << 15)] == want).all(), i


def test_norm_of_almost_2_31_rows(room):
    """The blocks' next row numbers pass 2^31."""
    room(100)
    c = AlmostTwoToThe31Rows()
    gamma, gs = torch.ones(c.k, dtype=torch.bfloat16, device="cuda"), dev_scalar(40.0)
    q, sf, _ = nv.add_rmsnorm_quant(c.x, gamma, 1e-6, gs=gs)
    want_q, want_sf, _ = nv.add_rmsnorm_quant(c.rows, gamma, 1e-6, gs=gs)
    c.check((q, want_q), (sf, want_sf))


def test_quantizers_of_almost_2_31_rows(room):
    """The warps' next task numbers pass 2^31 (MXFP4, the global scale's maximum)."""
    room(100)
    c = AlmostTwoToThe31Rows()
    c.x[-1, -1] = 100.0                                      # (the maximum is in the last task)
    assert float(nv.act_global_scale(c.x)[0]) == float(torch.tensor(2688.0 / 100.0))
    c.x[-1, -1] = c.rows[-1, -1]
    q, sf = nv.quant_act_mx(c.x)
    c.check(*zip((q, sf), nv.quant_act_mx(c.rows)))
    del q, sf
    gs = dev_scalar(40.0)
    q, sf = nv.quant_act(c.x, gs)
    c.check(*zip((q, sf), nv.quant_act(c.rows, gs)))
