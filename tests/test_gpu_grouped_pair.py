"""GPU tests of the grouped GEMM on CTA pairs (groups of 256 rows and more on
average, more tiles of 128 x 256 than SMs): groups whose last pair tile has one band, empty groups, output columns
that end inside a tile, unused bands before and after the groups, the largest
number of groups, agreement with the one-CTA kernel, and offsets that a kernel
before it on the stream has just written.

Tolerance against the 64-bit product, as for the GEMM epilogues: 2^-8 of the
value for the rounding to bf16, 1e-3 of the output's rms for the fp32 sums."""
import numpy as np
import pytest
import torch

import oracle
from _block_ref import activation, e4m3_value, f64, unpack_fp4
from _helpers import dev_scalar, nv, require_library, syn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def decode(packed, sf):
    return torch.from_numpy(unpack_fp4(packed) * np.repeat(e4m3_value(sf), 16, axis=1)).cuda()


def assert_close(got, ref, what):
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref) - 1.01 * 2.0 ** -8 * np.abs(ref)
    assert err.max() <= 1e-3 * np.sqrt((ref * ref).mean()), f"{what}: {err.max():.3e}"


def on_pairs(rows, groups, nw):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return rows >= 256 * groups and (rows + 127) // 128 * ((nw + 255) // 256) > sms


class Groups:
    """Operands of groups of the given rows, `lead` unused bands before them."""

    def __init__(self, group_m, nw, k, seed, lead=0, bias=True):
        self.group_m, self.nw, self.k, self.count = group_m, nw, k, len(group_m)
        bands = np.cumsum([lead] + [(m + 127) // 128 for m in group_m])
        self.offsets = (bands * 128).astype(np.int32)
        self.rows = int(self.offsets[-1])
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn(self.rows + 256, k, generator=g).bfloat16()
        self.w = (torch.randn(self.count * nw, k, generator=g) * 0.05).bfloat16()
        self.gx, self.gw = syn.global_scale(self.x), syn.global_scale(self.w)
        self.al = syn.alpha_of(self.gx, self.gw) * (1.0 + torch.arange(self.count) / 64.0).numpy()
        self.bias = torch.randn(self.count * nw, generator=g).bfloat16() if bias else None
        self.wq = nv.prepare_weight(self.w.cuda(), dev_scalar(self.gw))

    def run(self, act, rows):
        """Output [rows + 1, ldo] (its last row and columns past n as they were)."""
        n = self.nw // 2 if act in ("swiglu", "geglu") else self.nw
        x = torch.zeros(rows, self.k, dtype=torch.bfloat16)
        x[:self.x.shape[0]] = self.x[:rows]
        aq = nv.quant_act(x.cuda(), dev_scalar(self.gx))
        out = torch.full((rows + 1, n + 8), -5.0, dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_grouped_gemm_act(*aq, rows, torch.from_numpy(self.offsets).cuda(), self.count, *self.wq, n, self.k,
                                  torch.from_numpy(self.al.astype(np.float32)).cuda(),
                                  None if self.bias is None else self.bias.cuda(), nv.ACTIVATIONS[act], out, n + 8)
        torch.cuda.synchronize()
        nv.nvfp4_device_error()
        assert (out[:, n:] == -5.0).all() and (out[rows] == -5.0).all(), "written outside"
        return out[:, :n]

    def check(self, out, act, groups=None):
        got = f64(out)
        assert (got[:self.offsets[0]] == -5.0).all() and (got[self.offsets[-1]:] == -5.0).all(), "unused bands written"
        for g in range(self.count) if groups is None else groups:
            r = slice(int(self.offsets[g]), int(self.offsets[g]) + self.group_m[g])
            if self.group_m[g] == 0:
                continue
            w = slice(g * self.nw, (g + 1) * self.nw)
            v = decode(*oracle.quantize(syn.bf16_bits(self.x[r]), self.gx)) @ \
                decode(*oracle.quantize(syn.bf16_bits(self.w[w]), self.gw)).T
            v = v.cpu().numpy() * float(np.float32(self.al[g]))
            if self.bias is not None:
                v = v + f64(self.bias[w])
            assert_close(got[r], activation(v, act), f"group {g}")


@pytest.mark.parametrize("act,k", [("none", 264), ("none", 4104), ("relu", 2048), ("silu", 2056), ("swiglu", 2048),
                                   ("geglu", 4104)])
def test_ragged_groups(act, k):
    """Odd and even numbers of bands, empty groups first, last and between, one
    row, columns of 2176 weight rows (half of the last tile)."""
    c = Groups([0, 300, 257, 0, 1000, 1, 384, 513, 0], 2176, k, seed=5)
    rows = c.rows + 128
    assert on_pairs(rows, c.count, c.nw)
    c.check(c.run(act, rows), act)


def test_unused_bands_before_the_groups():
    c = Groups([200, 640], 3328, 512, seed=6, lead=3)
    assert on_pairs(c.rows + 256, c.count, c.nw)
    c.check(c.run("none", c.rows + 256), "none")


def test_no_rows_at_all():
    c = Groups([0, 0], 9984, 64, seed=7)
    assert on_pairs(512, c.count, c.nw)
    out = c.run("none", 256 * 2)
    assert (out == -5.0).all()


@pytest.mark.parametrize("count", [255, 256, 257])
def test_many_groups(count):
    """Up to 256 groups on pairs, more on the one-CTA kernel."""
    rng = np.random.default_rng(count)
    c = Groups([int(v) for v in rng.integers(0, 3, count) * 256 + rng.integers(0, 129, count)], 128, 64, seed=8)
    rows = max(c.rows, 256 * count)
    assert on_pairs(rows, count, c.nw)               # (by size; 257 groups are too many)
    c.check(c.run("none", rows), "none", groups=[0, 1, 7, 8, 31, 32, 100, 127, 128, 200, 247, 248, 253, count - 1])


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_same_as_the_one_cta_kernel(act):
    """The rows that the call is told of decide between the kernels: the same
    groups with and without a long unused end have the same bits."""
    c = Groups([300, 1, 100, 384, 128], 3456, 2048, seed=9)
    assert on_pairs(c.rows + 256, c.count, c.nw) and not on_pairs(c.rows, c.count, c.nw)
    a, b = c.run(act, c.rows), c.run(act, c.rows + 256)
    for g, m in enumerate(c.group_m):
        r = slice(int(c.offsets[g]), int(c.offsets[g]) + m)
        assert torch.equal(a[r].view(torch.int16), b[r].view(torch.int16)), f"group {g}"


def test_offsets_from_the_kernel_before():
    """Sort, dispatch and GEMM in turn on the same buffers without a
    synchronisation, another routing each time."""
    tokens, topk, experts, h, n = 1500, 2, 8, 512, 1280
    g = torch.Generator(device="cuda").manual_seed(10)
    x = torch.randn(tokens, h, device="cuda", generator=g).bfloat16()
    wq = nv.prepare_weight((torch.randn(experts * n, h, device="cuda", generator=g) * 0.05).bfloat16(), dev_scalar(40.0))
    al = torch.full((experts,), 1e-4, device="cuda")
    rows = nv.nvfp4_moe_rows(tokens, topk, experts)
    assert on_pairs(rows, experts, n)
    kp = nv.padded_k(h)
    q = torch.zeros(rows, kp // 2, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(nv.nvfp4_scale_bytes(rows, h), dtype=torch.uint8, device="cuda")
    ws = torch.empty(max(1, nv.nvfp4_moe_sort_workspace_bytes(tokens, topk, experts)), dtype=torch.uint8, device="cuda")
    off = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    cnt = torch.empty(experts, dtype=torch.int32, device="cuda")
    dest = torch.empty(tokens, topk, dtype=torch.int32, device="cuda")
    gs = dev_scalar(40.0)
    ids = [torch.randint(0, 1 + i % experts, (tokens, topk), device="cuda", generator=g, dtype=torch.int32)
           for i in range(12)]
    torch.cuda.synchronize()

    def layer(i, out, sync):
        wait = torch.cuda.synchronize if sync else (lambda: None)
        nv.nvfp4_moe_sort(ids[i], 4, tokens, topk, experts, off, cnt, dest, ws, ws.numel())
        wait()
        nv.nvfp4_moe_dispatch_quant(x, h, gs, dest, tokens, topk, rows, h, q, sf)
        wait()
        nv.nvfp4_grouped_gemm(q, sf, rows, off, experts, *wq, n, h, al, None, out, n)
        wait()
        got = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_moe_combine(out, n, None, dest, tokens, topk, rows, n, None, 0, got, n)
        return got

    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    quick = [layer(i, out, False) for i in range(12)]
    torch.cuda.synchronize()
    slow = [layer(i, out, True) for i in range(12)]
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    for i in range(12):
        assert torch.equal(quick[i].view(torch.int16), slow[i].view(torch.int16)), i
