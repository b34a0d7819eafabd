"""GPU tests of the norm's persistent kernel, which takes over where there are more rows
than resident blocks: its ring goes round several times, rows end anywhere inside a copied
piece, a thread owns one or two steps of a row, blocks differ in their number of rows, and h
may replace x or the residual while later rows are already being copied.  Definition and
bounds as in the tests of the norm's other kernel."""
import numpy as np
import pytest
import torch

import oracle
from _block_ref import FMT_MXFP4, FMT_MXFP8, FMT_NVFP4
from _helpers import dev_scalar, nv, require_library
from test_gpu_norm_quant import ALL, EPS, _check, _run, _strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def resident_rows(k, res):
    """Rows that the persistent kernel works on at once (blocks per SM by their threads and by
    two rows of shared memory each, times the SMs), None where it does not take such rows."""
    units = (k + 15) // 16
    steps = 1 if units <= 512 else 2 if units <= 1024 else 4
    threads = ((units + steps - 1) // steps + 31) // 32 * 32
    stage = (k + 7) // 8 * 16 * (2 if res else 1)
    blocks = max(1, min(32, (1024 if steps == 1 else 512) // threads))
    fitting = lambda n: (224 * 1024 - n * 1536) // n // stage  # noqa: E731
    while blocks > 1 and fitting(blocks) < 2:
        blocks -= 1
    if steps > 2 or fitting(blocks) < 2:
        return None
    return blocks * torch.cuda.get_device_properties(0).multi_processor_count


def rounds(m, k, res):
    """How often the blocks with the most rows go on to another row."""
    return (m - 1) // resident_rows(k, res)


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("k", [8, 520, 2056, 5128])
def test_one_step_rows(k, res, fmt):
    """Five rounds and a partial one: more than the ring's four stages."""
    m = 5 * resident_rows(k, res) + 77
    assert rounds(m, k, res) == 5
    _run(m, k, fmt, pad=8 if k > 8 else 0, res=res, seed=k + res)


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("k,res", [(8200, True), (14336, False), (16384, True)])
def test_two_step_rows(k, res, fmt):
    m = 5 * resident_rows(k, res) + 3
    assert rounds(m, k, res) == 5
    _run(m, k, fmt, res=res, seed=k)


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("k", [1, 17, 31, 33, 1000, 1021, 8201])
def test_row_ends_inside_a_copied_piece(k, fmt):
    """The strides, not the lengths, are multiples of 8; what follows a row's end is NaN."""
    m = 2 * resident_rows(k, False) + 19
    assert rounds(m, k, False) == 2
    _run(m, k, fmt, pad=(-k) % 8 + 8, res=False, seed=k)


@pytest.mark.parametrize("in_place", ["x", "residual"])
@pytest.mark.parametrize("k", [264, 4096])
def test_in_place_under_look_ahead(k, in_place):
    """h over its own row's x or residual; the next rows' copies are in flight."""
    m = 6 * resident_rows(k, True) + 1
    assert rounds(m, k, True) == 6
    _run(m, k, FMT_NVFP4, seed=k, in_place=in_place)


def test_the_switch_between_the_kernels():
    """As many rows as blocks (a block per row), and one more (the ring)."""
    k = 1032
    n = resident_rows(k, True)
    x, r = _strided(n + 1, k, 0, 51), _strided(n + 1, k, 0, 52)
    gamma = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    for fmt in ALL:
        gs = dev_scalar(40.0) if fmt == FMT_NVFP4 else None
        a = nv.add_rmsnorm_quant(x[:n], gamma, EPS, residual=r[:n], gs=gs, fmt=fmt)
        b = nv.add_rmsnorm_quant(x, gamma, EPS, residual=r, gs=gs, fmt=fmt)
        torch.cuda.synchronize()
        _check(x[:n], r[:n], gamma, fmt, 40.0, *a)
        _check(x, r, gamma, fmt, 40.0, *b)


def test_rows_of_zeros_and_non_finite_rows_between_others():
    k = 1032
    n = resident_rows(k, False)
    m = 3 * n + 5
    x = _strided(m, k, 8, 61)
    bad = [3, n + 3, 2 * n, m - 1]                           # the rows before and after them in a block, too
    zero = [0, 2 * n + 3, m - 2]
    clean = x.clone()
    x[zero] = clean[zero] = 0
    x[bad[:2], 5] = float("nan")
    x[bad[2:], k - 1] = float("inf")
    gamma = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    good = np.setdiff1d(np.arange(m), bad)
    for fmt in (FMT_NVFP4, FMT_MXFP4, FMT_MXFP8):
        gs = dev_scalar(40.0) if fmt == FMT_NVFP4 else None
        got_q, got_sf, _ = nv.add_rmsnorm_quant(x, gamma, EPS, gs=gs, fmt=fmt)
        want_q, want_sf, _ = nv.add_rmsnorm_quant(clean, gamma, EPS, gs=gs, fmt=fmt)
        torch.cuda.synchronize()
        _check(clean, None, gamma, fmt, 40.0, want_q, want_sf, None)
        assert torch.equal(got_q[good], want_q[good])
        cols = nv.padded_k(k) // (16 if fmt == FMT_NVFP4 else 32)
        a, b = (oracle.unswizzle(t.cpu().numpy(), m, (cols + 3) // 4 * 4) for t in (got_sf, want_sf))
        assert np.array_equal(a[good], b[good])


def test_repeats_bit_for_bit_on_another_stream():
    x, r = _strided(4000, 2048, 0, 71), _strided(4000, 2048, 0, 72)
    assert rounds(4000, 2048, True) >= 3
    gamma = torch.full((2048,), 1.25, dtype=torch.bfloat16, device="cuda")
    a = nv.add_rmsnorm_quant(x, gamma, EPS, residual=r, gs=dev_scalar(40.0))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = nv.add_rmsnorm_quant(x, gamma, EPS, residual=r, gs=dev_scalar(40.0))
    s.synchronize()
    nv.nvfp4_device_error()
    assert all(torch.equal(i, j) for i, j in zip(a, b))
