"""GPU tests of the weight gradient from 8-bit checkpoints against the 64-bit product.

The products are exact.  Sums in fp32 on the tensor cores: a step adds 16 rows to the sum,
each addition off by at most 2^-22 (a truncated ulp and as much for aligning the 16) of the
magnitudes' sum: (rows / 16 + 1) 2^-22 of it.  bf16 results add half a step, 2^-8."""
import numpy as np
import pytest
import torch

import _train_ref as ref
from _helpers import nv, require_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def operands(rows, n, k, seed, pad=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dy = (torch.randn(rows, (n + 7) // 8 * 8 + pad, device="cuda", generator=g) * 0.1).to(torch.bfloat16)[:, :n]
    x = torch.randn(rows, (k + 7) // 8 * 8, device="cuda", generator=g) * std
    x[:, ::29] *= 30
    _, q, sf = nv.act_checkpoint(x.to(torch.bfloat16)[:, :k])
    torch.cuda.synchronize()
    return dy, q, sf, torch.from_numpy(ref.decode(q, sf, rows, k)).cuda()


def assert_close(got, dy, x, rows):
    want, mag = dy.double().T @ x, dy.double().abs().T @ x.abs()
    tol = (rows / 16 + 1) * 2.0 ** -22 * mag
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    err = (got.double() - want).abs()
    assert bool((err <= tol + 2.0 ** -126).all()), float((err / tol.clamp_min(1e-300)).max())
    return float((got.double() - want).norm() / want.norm().clamp_min(1e-300))


SHAPES = [(1, 1, 1), (1, 8, 8), (1, 300, 700), (16, 17, 33), (63, 256, 256), (64, 256, 256), (65, 300, 260), (128, 128, 128),
          (200, 129, 136), (333, 2072, 520), (1000, 520, 1000), (2049, 264, 128), (96, 1000, 4104),
          (1100, 2600, 2570), (20000, 100, 70), (3333, 300, 261)]     # parts of a sum, ranges of the rows


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_dense(m, n, k, dtype):
    dy, q, sf, x = operands(m, n, k, m + n + k, pad=8)
    dw = nv.checkpoint_wgrad(dy, q, sf, k, dtype=dtype)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    assert dw.shape == (n, k)
    assert_close(dw, dy, x, m)


@pytest.mark.parametrize("m", [150, 1500, 12000])
def test_columns_past_k_and_accumulation(m):
    n, k = 70, 45
    dy, q, sf, x = operands(m, n, k, 1)
    buf = torch.full((n, 64), 5.0, device="cuda")
    base = torch.randn(n, k, device="cuda")
    buf[:, :k] = base
    nv.checkpoint_wgrad(dy, q, sf, k, dw=buf[:, :k], accumulate=True)
    plain = nv.checkpoint_wgrad(dy, q, sf, k)
    torch.cuda.synchronize()
    # (the sums of parts and ranges meet dw one after the other: a rounding each)
    assert (buf[:, :k] - (base + plain)).abs().max() <= 16 * 2.0 ** -24 * (base.abs() + 2 * plain.abs()).max()
    assert m > 512 or torch.equal(buf[:, :k], base + plain)
    assert (buf[:, k:] == 5).all()
    half = torch.full((n, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    nv.checkpoint_wgrad(dy, q, sf, k, dw=half[:, :k])
    torch.cuda.synchronize()
    assert torch.equal(half[:, :k], plain.to(torch.bfloat16)) and (half[:, k:] == 5).all()


def test_no_rows():
    dy, q, sf, _ = operands(4, 40, 50, 2)
    empty = dy[:0], q[:0], sf
    dw = torch.full((40, 56), 5.0, device="cuda")
    nv.checkpoint_wgrad(*empty, 50, dw=dw[:, :50], accumulate=True)
    torch.cuda.synchronize()
    assert (dw == 5).all()
    nv.checkpoint_wgrad(*empty, 50, dw=dw[:, :50])
    torch.cuda.synchronize()
    assert (dw[:, :50] == 0).all() and (dw[:, 50:] == 5).all()


@pytest.mark.parametrize("std", [2.0 ** -100, 2.0 ** -20, 2.0 ** 15, 2.0 ** 60])
def test_scales_over_the_whole_range(std):
    """Scale codes on both sides of where one bf16 factor is enough."""
    dy, q, sf, x = operands(80, 64, 96, 3, std=std)
    dw = nv.checkpoint_wgrad(dy, q, sf, 96)
    torch.cuda.synchronize()
    assert_close(dw, dy, x, 80)


def test_every_code_is_exact():
    """x one-hot rows of dy: dw is x itself.  All 254 finite codes at scales 2^-127 .. 2^119."""
    codes = torch.arange(256, dtype=torch.int32)
    codes = codes[(codes & 127) != 127]
    for exps in (range(-127, -60), range(-60, 8), range(8, 120)):
        exps = list(exps)
        q = codes.to(torch.uint8).repeat(len(exps), 1)
        q = torch.nn.functional.pad(q, (0, 256 - q.shape[1])).cuda()
        rows = len(exps)
        sf = torch.zeros((rows + 127) // 128 * 128, 8, dtype=torch.uint8)
        sf[:rows] = torch.tensor([e + 127 for e in exps], dtype=torch.uint8)[:, None]
        flat = sf.view(-1, 4, 32, 2, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous().cuda()
        dy = torch.eye(rows, (rows + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")[:, :rows]
        dw = nv.checkpoint_wgrad(dy, q, flat, 256)
        torch.cuda.synchronize()
        want = ref.decode(q, flat, rows, 256)
        got = dw.double().cpu().numpy()
        normal = np.abs(want) >= 2.0 ** -126
        assert np.array_equal(got[normal], want[normal])
        assert np.all(np.abs(got - want)[~normal] <= 2.0 ** -126)


def test_nan_blocks_show():
    dy, q, sf, _ = operands(40, 32, 64, 4)
    x = torch.randn(40, 64, device="cuda").to(torch.bfloat16)
    x[7, 33] = float("inf")
    _, q, sf = nv.act_checkpoint(x)
    dw = nv.checkpoint_wgrad(dy, q, sf, 64)
    torch.cuda.synchronize()
    assert torch.isnan(dw[:, 32:]).all() and torch.isfinite(dw[:, :32]).all()


@pytest.mark.parametrize("scale", [127, 200])
def test_nan_codes_show(scale):
    """E4M3's NaN, of either sign, in any place of a word."""
    dy, q, sf, _ = operands(70, 32, 64, 4)
    sf.fill_(scale)
    q.fill_(0x30)
    for i, (row, col) in enumerate([(0, 0), (3, 9), (31, 18), (64, 27), (69, 63), (5, 36)]):
        q[row, col] = 0x7F if i % 2 else 0xFF
    dw = nv.checkpoint_wgrad(dy, q, sf, 64)
    torch.cuda.synchronize()
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[0, 9, 18, 27, 36, 63]] = True
    assert torch.isnan(dw[:, bad]).all() and torch.isfinite(dw[:, ~bad]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts", [[5], [0, 0], [1, 0, 130, 128], [127, 1, 0, 64, 65, 300, 0], [64] * 9, [2100, 0, 1025]])
@pytest.mark.parametrize("n,k", [(128, 64), (300, 300)])
def test_groups(counts, n, k, dtype):
    """Padding rows of both operands hold NaN."""
    offsets, cnt, rows, real = ref.groups_of(counts)
    dy, q, sf, x = operands(rows, n, k, 5)
    keep = torch.from_numpy(real).cuda()
    dy[~keep] = float("nan")
    q[~keep] = 0x7F
    dw = nv.checkpoint_wgrad(dy, q, sf, k, offsets, cnt, dtype=dtype)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    dw = dw.view(len(counts), n, k)
    for g, c in enumerate(counts):
        o = int(offsets[g])
        assert_close(dw[g], dy[o:o + c], x[o:o + c], c)
        if c == 0:
            assert (dw[g] == 0).all()
    more = torch.ones(len(counts) * n, (k + 7) // 8 * 8, device="cuda")[:, :k]
    if dtype == torch.float32:
        nv.checkpoint_wgrad(dy, q, sf, k, offsets, cnt, dw=more, accumulate=True)
        torch.cuda.synchronize()
        assert torch.allclose(more.view_as(dw), dw + 1, rtol=0, atol=4 * 2.0 ** -24 * float(dw.abs().max() + 1))
        assert max(counts) > 1024 or torch.equal(more.view_as(dw), dw + 1)


def test_repeats_give_the_same_bits():
    for m, n, k in ((3000, 520, 260), (3000, 2200, 2400)):
        dy, q, sf, _ = operands(m, n, k, 6)
        first = nv.checkpoint_wgrad(dy, q, sf, k)
        for _ in range(4):
            assert torch.equal(first, nv.checkpoint_wgrad(dy, q, sf, k))


def test_captured_and_on_another_stream():
    dy, q, sf, x = operands(500, 264, 130, 7)
    dw = torch.zeros(264, 136, device="cuda")[:, :130]
    ws = torch.zeros(nv.nvfp4_checkpoint_wgrad_workspace_bytes(500, 264, 130), dtype=torch.uint8, device="cuda")

    def step():
        nv.checkpoint_wgrad(dy, q, sf, 130, dw=dw, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (8, 9):
        dy2, q2, sf2, x2 = operands(500, 264, 130, seed)
        dy.copy_(dy2), q.copy_(q2), sf.copy_(sf2)
        graph.replay()
        torch.cuda.synchronize()
        assert_close(dw, dy, x2, 500)


@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_a_call_belongs_to_its_stream(handle):
    """The stream of the call lags behind the current one, then the current one behind it."""
    m, n, k = 4096, 256, 256
    dy, q, sf, _ = operands(m, n, k, 12)
    want = nv.checkpoint_wgrad(dy, q, sf, k)
    size = nv.nvfp4_checkpoint_wgrad_workspace_bytes(m, n, k)
    assert size >= 8 * n * k * 4
    s = torch.cuda.Stream()
    arg = s.cuda_stream if handle else s
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    got = nv.checkpoint_wgrad(dy, q, sf, k, stream=arg)      # its workspace is free again before it ran
    later = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all((t == 255).all() for t in later)
    before = [torch.empty(n, k, device="cuda") for _ in range(4)]
    torch.cuda._sleep(20_000_000)
    for t in before:
        t.fill_(7.0)
    del t, before                                            # free for the current stream's next tensors only
    got = nv.checkpoint_wgrad(dy, q, sf, k, stream=arg)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    nv.nvfp4_device_error()


def test_calls_on_two_streams_at_once():
    """Split rows, whole rounds of tiles and groups, interleaved."""
    offsets, cnt, rows, _ = ref.groups_of([300, 0, 129, 1000])
    calls = []
    for i, (m, n, k, groups) in enumerate([(4096, 256, 256, ()), (700, 2600, 2100, ()), (rows, 512, 300, (offsets, cnt))]):
        dy, q, sf, _ = operands(m, n, k, 20 + i)
        calls.append((dy, q, sf, k, *groups))
    want = [nv.checkpoint_wgrad(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[nv.checkpoint_wgrad(*calls[(i + j) % 3], stream=s) for j, s in enumerate(streams)] for i in range(9)]
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    for i, pair in enumerate(got):
        for j, dw in enumerate(pair):
            assert torch.equal(dw, want[(i + j) % 3])


def test_error_of_long_sums(capsys):
    """8192 rows: within the bound, and printed for the record."""
    dy, q, sf, x = operands(8192, 256, 256, 10)
    rel = assert_close(nv.checkpoint_wgrad(dy, q, sf, 256), dy, x, 8192)
    with capsys.disabled():
        print(f" [relative error of fp32 sums of 8192 rows: {rel:.2e}]", end="")
