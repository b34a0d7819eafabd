"""GPU tests of the quantizing norm against its definition in 64 bits.

Bounds.  The kernel's y differs from the exact one by the rounding of fp32
sums and products only.  A row's sum of squares has at most 64 terms per
thread, 5 shuffles and 32 warps in a chain: relative error below
(64 + 5 + 32 + 2) 2^-24; its square root halves that; the division, root and
two products add at most 4 more 2^-24.  The residual's addition in fp32 adds one
rounding of h, so DELTA = (52 + 4 + 4) 2^-24 < 4e-6 covers y.  A code is right if
it lies between the codes of y (1 - DELTA) and y (1 + DELTA) under the kernel's
own block scale, and a scale if it lies between those of amax (1 -+ DELTA).
Where the addition cancels, h itself carries 2^-24 of |x| + |r|: the tests' h
is taken as the fp32 sum, which the format of the inputs makes exact to state."""
import numpy as np
import pytest
import torch

from _block_ref import FMT_MXFP4, FMT_MXFP8, FMT_NVFP4, bf16_round, e2m1, e4m3, e4m3_value, f64, floor_log2, unpack_fp4, untile
from _helpers import dev_scalar, nv, require_library, syn

pytestmark = pytest.mark.gpu
DELTA = 4e-6
EPS = 1e-6
ALL = [FMT_NVFP4, FMT_MXFP4, FMT_MXFP8]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def _strided(m, k, pad, seed, make=syn.bf16_outlier_channels):
    full = torch.zeros((m, k + pad), dtype=torch.bfloat16)
    full[:, :k] = make(m, k, seed)
    full[:, k:] = float("nan")                                # never read
    return full.cuda()[:, :k]


def _between(code, f, v):
    lo, hi = f(np.abs(v) * (1 - DELTA)), f(np.abs(v) * (1 + DELTA))
    return (np.abs(code) >= lo) & (np.abs(code) <= hi)


def _check(x, r, gamma, fmt, gs, x_q, x_sf, h, rows=None):
    m, k = x.shape
    kp = nv.padded_k(k)
    hx = (x.float() + r.float()).cpu() if r is not None else x.float().cpu()
    if h is not None:
        assert torch.equal(h.cpu(), hx.to(torch.bfloat16)), "h"
    h64 = hx.double().numpy()
    y = h64 / np.sqrt(np.mean(h64 * h64, axis=1, keepdims=True) + EPS) * f64(gamma)
    y = np.pad(y, ((0, 0), (0, kp - k)))
    blk = 16 if fmt == FMT_NVFP4 else 32
    sf, full = untile(x_sf.cpu().numpy(), m, kp // blk)
    pad = full.copy()
    pad[:m, :kp // blk] = 0
    assert not pad.any(), "scale padding is not zero"
    amax = np.abs(y.reshape(m, -1, blk)).max(-1)
    q = e4m3_value(x_q.cpu().numpy()) if fmt == FMT_MXFP8 else unpack_fp4(x_q.cpu().numpy())
    sel = slice(None) if rows is None else rows
    if fmt == FMT_NVFP4:
        scale = e4m3_value(sf)
        ok = _between(scale, lambda a: e4m3(a * gs / 6.0), amax)
        inv = np.divide(gs, scale, out=np.zeros_like(scale), where=scale > 0)
    else:
        emax = 8 if fmt == FMT_MXFP8 else 2
        code = lambda a: np.where(a > 0, np.clip(floor_log2(np.maximum(a, 1e-300)) - emax, -127, 127), -127) + 127  # noqa: E731
        ok = _between(sf.astype(np.int64), code, amax)
        inv = 2.0 ** (127.0 - sf.astype(np.float64))
    assert ok[sel].all(), "block scales"
    v = y * np.repeat(inv, blk, axis=1)
    ok = _between(q, e4m3 if fmt == FMT_MXFP8 else e2m1, v) & ((q == 0) | (np.sign(q) == np.sign(v)))
    assert ok[sel].all(), f"{(~ok[sel]).sum()} codes"


def _run(m, k, fmt, pad=0, res=True, seed=0, make=syn.bf16_outlier_channels, gs=40.0, in_place=None):
    x = _strided(m, k, pad, seed, make)
    r = _strided(m, k, 8, seed + 1) if res else None
    gamma = (1.0 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).cuda()
    g = dev_scalar(gs) if fmt == FMT_NVFP4 else None
    x0, r0 = x.clone(), r.clone() if res else None
    h = {None: None, "x": x, "residual": r}[in_place]
    x_q, x_sf, h = nv.add_rmsnorm_quant(x, gamma, EPS, residual=r, gs=g, fmt=fmt, h=h)
    torch.cuda.synchronize()
    assert (h is None) == (not res)
    _check(x0, r0, gamma, fmt, gs, x_q, x_sf, h)


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("m,k", [(1, 4096), (1, 8), (3, 40), (129, 256), (5, 5128), (2, 8200), (7, 14336)])
def test_shapes(m, k, fmt):
    _run(m, k, fmt, seed=m + k)


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("k", [1, 17, 31, 33, 1000, 16392, 65536])
def test_row_ends_inside_a_vector_or_takes_many_steps(k, fmt):
    """Rows of any length; the strides (not the lengths) are multiples of 8."""
    _run(3, k, fmt, pad=(-k) % 8 + 8, res=False, seed=k)


@pytest.mark.parametrize("in_place", ["x", "residual"])
def test_in_place_residual_stream(in_place):
    _run(200, 2080, FMT_NVFP4, seed=11, in_place=in_place)


def test_many_rows_strided():
    _run(1025, 520, FMT_MXFP8, pad=56, seed=12)


def test_zero_rows_and_tiny_values():
    """All-zero rows give zero codes and scales (eps keeps the norm finite); a
    row of values far below eps is scaled by 1 / sqrt(eps)."""
    make = lambda m, k, seed: torch.cat([torch.zeros(2, k), torch.full((m - 2, k), 2.0 ** -60)]).to(torch.bfloat16)  # noqa: E731
    for fmt in ALL:
        _run(4, 96, fmt, res=False, make=make)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_row_leaves_the_others_alone(bad):
    m, k = 6, 320
    x = _strided(m, k, 0, 21)
    x[2, 5] = bad
    gamma = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    for fmt in ALL:
        x_q, x_sf, _ = nv.add_rmsnorm_quant(x, gamma, EPS, gs=dev_scalar(40.0), fmt=fmt)
        torch.cuda.synchronize()
        good = [i for i in range(m) if i != 2]
        # only the good rows' values are compared; the bad row's are unspecified
        clean = x.clone()
        clean[2] = 0
        x_q[2] = 0
        sf = x_sf.clone()
        _check_rows(clean, gamma, fmt, x_q, sf, good)


def _check_rows(x, gamma, fmt, x_q, x_sf, good):
    kp = nv.padded_k(x.shape[1])
    blk = 16 if fmt == FMT_NVFP4 else 32
    sub_q = x_q[good]
    lin, _ = untile(x_sf.cpu().numpy(), x.shape[0], kp // blk)
    want_q, want_sf, _ = nv.add_rmsnorm_quant(x[good], gamma, EPS, gs=dev_scalar(40.0), fmt=fmt)
    torch.cuda.synchronize()
    want, _ = untile(want_sf.cpu().numpy(), len(good), kp // blk)
    assert torch.equal(sub_q, want_q) and np.array_equal(lin[good], want)


def test_feeds_the_gemm_like_the_separate_steps():
    """norm -> NVFP4 -> GEMM equals the GEMM of the codes decoded in 64 bits."""
    m, k, n = 48, 1024, 256
    x, r = _strided(m, k, 0, 31), _strided(m, k, 0, 32)
    gamma = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    w = syn.bf16_normal((n, k), 0.02, 33)
    gw = syn.global_scale(w)
    w_fp4, w_sf = nv.prepare_weight(w.cuda(), dev_scalar(gw))
    gs = 60.0
    x_q, x_sf, h = nv.add_rmsnorm_quant(x, gamma, EPS, residual=r, gs=dev_scalar(gs))
    out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_gemm(x_q, x_sf, m, w_fp4, w_sf, n, n, k, dev_scalar(syn.alpha_of(gs, gw)), None, out, n)
    torch.cuda.synchronize()
    deq = lambda q, sf, rows: unpack_fp4(q.cpu().numpy()) * np.repeat(e4m3_value(untile(sf.cpu().numpy(), rows, k // 16)[0]), 16, 1)  # noqa: E731
    ref = deq(x_q, x_sf, m) @ deq(w_fp4, w_sf, n).T * syn.alpha_of(gs, gw)
    assert np.abs(f64(out) - ref).max() <= 2e-2 * np.sqrt((ref * ref).mean())


def test_side_stream_and_repeat():
    """Work goes to the stream that is current; the same call twice gives the same bytes."""
    x, r = _strided(300, 4096, 0, 41), _strided(300, 4096, 0, 42)
    gamma = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    a = nv.add_rmsnorm_quant(x, gamma, EPS, residual=r, fmt=FMT_MXFP8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = nv.add_rmsnorm_quant(x, gamma, EPS, residual=r, fmt=FMT_MXFP8)
    s.synchronize()
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_empty_call():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    x_q, _, _ = nv.add_rmsnorm_quant(x, torch.ones(64, dtype=torch.bfloat16, device="cuda"), EPS, fmt=FMT_MXFP8)
    assert x_q.shape == (0, 64)


def test_bf16_round_helper():
    assert bf16_round(np.float32(1.00390625)) == 1.0       # a tie goes to the even bf16
