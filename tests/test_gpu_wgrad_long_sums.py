"""GPU tests of weight gradients over many rows, whose sums are made of parts: 2048 rows into fp32 gradients,
8192 into bf16 ones."""
import pytest
import torch

import _train_ref as ref
from _helpers import nv, require_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def operands(rows, n, k, seed, positive=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def new(cols, std):                                      # rows on 16-byte boundaries
        t = (torch.randn(rows, (cols + 7) // 8 * 8, device="cuda", generator=g) * std).to(torch.bfloat16)
        return (t.abs() if positive else t)[:, :cols]

    dy, x = new(n, 0.1), new(k, 1.0)
    _, q, sf = nv.act_checkpoint(x)
    return dy, q, sf


def gradient(dy, q, sf, k, groups, dtype=torch.float32):
    dw = nv.checkpoint_wgrad(dy, q, sf, k, *groups, dtype=dtype)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    return dw


@pytest.mark.parametrize("rows", [65536, 262144])
def test_a_bf16_gradient_falls_no_shorter_the_more_rows_it_has(rows):
    """Sums of one sign.  A step of 16 rows takes at most 2^-23 of the sum so far: half of 512 steps of it over
    the 8192 rows of a part, 2^-15, and over 262144 rows in one sum 2^-10.  The fp32 gradient is off by at most a
    quarter of that and rounded alike, so that the mean over 65536 elements shows the difference alone."""
    offsets, cnt, m, _ = ref.groups_of([rows])
    dy, q, sf = operands(m, 256, 256, 1, positive=True)
    want = gradient(dy, q, sf, 256, (offsets, cnt)).double()
    got = gradient(dy, q, sf, 256, (offsets, cnt), torch.bfloat16).double()
    rounded = want.to(torch.bfloat16).double()
    assert float(((got - rounded) / want).mean().abs()) <= 2.0 ** -15 * (1 + 1 / 4) + 1e-5


@pytest.mark.parametrize("m,n,k,counts", [
    (40000, 2600, 2570, None),                              # 121 tiles: a pair has another one after
    (8193, 2560, 2600, None), (24576, 2600, 2560, None),
    (0, 300, 264, [20000, 100, 0, 8192, 8193, 3000, 16500]),
    (0, 1500, 1500, [8200, 5, 0, 300, 16385, 64])])         # 216 tiles: a pair has long, short and empty sums in a row
def test_parts_of_bf16_gradients(m, n, k, counts):
    """Against the fp32 gradient: half a step of bf16, and the steps' bound for the rows of a part."""
    groups = ()
    if counts:
        *groups, m, real = ref.groups_of(counts)
    dy, q, sf = operands(m, n, k, 2)
    mag = gradient(*operands(m, n, k, 2, positive=True), k, groups).double()
    if counts:
        dy[~torch.from_numpy(real).cuda()] = float("nan")
    want = gradient(dy, q, sf, k, groups).double()
    got = gradient(dy, q, sf, k, groups, torch.bfloat16).double()
    tol = 1.001 * (8192 / 16 + 1) * 2.0 ** -22 * mag
    assert bool(((got - want).abs() <= 2.0 ** -8 * (want.abs() + tol) + tol).all())
    assert torch.equal(got, gradient(dy, q, sf, k, groups, torch.bfloat16).double())


def test_accumulation_of_long_sums_adds_once():
    """dw + the sum of all parts, rounded once."""
    offsets, cnt, m, _ = ref.groups_of([7000, 0, 2048, 4097])
    dy, q, sf = operands(m, 300, 264, 3)
    groups = offsets, cnt
    base = torch.randn(4 * 300, 264, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    dw = base.clone()
    nv.checkpoint_wgrad(dy, q, sf, 264, *groups, dw=dw, accumulate=True)
    assert torch.equal(dw, base + gradient(dy, q, sf, 264, groups))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_last_part_before_the_most_rows(dtype):
    """2^31 - 1024 rows in one group (a part further on the row number would leave 32 bits), 112 GB: all but
    some rows are zero."""
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 112 GB")
    rows, n, k = (1 << 31) - 1024, 8, 32
    dy = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    sf = torch.full((nv.nvfp4_mxfp4_scale_bytes(rows, k),), 127, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    want = torch.zeros(n, k, dtype=torch.float64, device="cuda")
    for at in (0, 1 << 30, rows - 64):
        dy[at:at + 64] = torch.randint(-4, 5, (64, n), device="cuda", generator=g).to(torch.bfloat16)
        codes = torch.randint(0, 0x39, (64, k), device="cuda", generator=g).to(torch.uint8)
        q[at:at + 64] = codes
        want += dy[at:at + 64].double().T @ codes.view(torch.float8_e4m3fn).double()
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    got = gradient(dy, q, sf, k, (offsets, offsets[1:].contiguous()), dtype).double()
    tol = 192 * 4 * 2.0 ** -22                               # (of at most 192 products of up to 4; zeros add nothing)
    assert bool(((got - want).abs() <= tol + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0)).all())


@pytest.mark.parametrize("n,k", [(256, 256), (300, 333)])
def test_parts_keep_the_error_of_an_fp32_gradient(n, k):
    """One group of 8192 rows of both signs: off by 6e-7 with parts of 2048 rows, 3.5e-6 in one sum."""
    offsets, cnt, rows, _ = ref.groups_of([8192])
    dy, q, sf = operands(rows, n, k, 6)
    want = dy[:8192].double().T @ torch.from_numpy(ref.decode(q, sf, rows, k)[:8192]).cuda()
    got = gradient(dy, q, sf, k, (offsets, cnt))
    assert float((got.double() - want).norm() / want.norm()) <= 1.5e-6
