"""GPU tests of the 8-bit activation checkpoints and the activation's gradient.

Codes and scales of x are exact.  The activation in fp32: its exponential's argument is
rounded to 2^-22 of itself, so for |argument| <= 64 act and slope are within 2^-15 of their terms; bf16
outputs add half a step, 2^-8.  Where the exponential would leave the floats, arguments below -87, the
sigmoid is below 2^-125 and may be taken for 0 or held there: |v sigmoid| <= 87.4 * 2^-125.5 < 2^-119 (it falls
beyond), so that either way act is off by less than 2^-118, and a gated one by that times up (TINY)."""
import numpy as np
import pytest
import torch

import _train_ref as ref
from _block_ref import e4m3_value, untile
from _helpers import nv, require_library

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "silu", "swiglu", "geglu"]
EPS = 2.0 ** -15
HALF = 2.0 ** -8 * (1 + 2.0 ** -8)                           # half a step of bf16


def tiny(*factors):
    return 2.0 ** -118 * np.prod([1 + np.abs(f).max() for f in factors])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def bf16(rows, cols, seed, std=1.5, pad=0):
    """[rows, cols] bf16, rows on 16-byte boundaries; blocks of very different size, zeros among them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, (cols + 7) // 8 * 8 + pad, device="cuda", generator=g) * std
    x[:, ::37] *= 20
    x[rows // 2, :] = 0
    return x.to(torch.bfloat16)[:, :cols]


def columns(n, act):
    return 2 * n if act in ("swiglu", "geglu") else n


def assert_codes(q, sf, v, rows, cols):
    """Exactly the codes and scales of v; -0 and 0 alike."""
    want, s = ref.mxfp8(v)
    got = e4m3_value(q.cpu().numpy().reshape(rows, -1))
    assert np.array_equal(got, want)
    kp = (cols + 31) // 32 * 32
    codes, full = untile(sf.cpu().numpy(), rows, kp // 32)
    assert np.array_equal(codes, s)
    pad = full.copy()
    pad[:rows, :kp // 32] = 0
    assert not pad.any()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n", [(1, 1), (1, 8), (3, 16), (2, 33), (5, 100), (129, 64), (7, 520), (40, 1000), (2, 4104),
                                 (3, 9000)])
def test_forward(m, n, act):
    k = columns(n, act)
    x = bf16(m, k, m + n, pad=8)
    out, q, sf = nv.act_checkpoint(x, act)
    torch.cuda.synchronize()
    v = ref.f64(x)
    assert_codes(q, sf, v, m, k)
    if act == "none":
        assert out is None
        return
    want = ref.forward(v, act)
    assert np.all(np.abs(ref.f64(out) - want) <= HALF * np.abs(want) + tiny(v))


def test_forward_of_none_copies():
    x, out = bf16(9, 40, 1), torch.zeros(9, 40, dtype=torch.bfloat16, device="cuda")
    got, q, sf = nv.act_checkpoint(x, "none", out=out)
    assert got is out and torch.equal(out, x)
    a = nv.act_checkpoint(x)
    assert torch.equal(a[1], q) and torch.equal(a[2], sf)


def test_wide_range_of_blocks_and_non_finite_ones():
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    x[0, :32] = 2.0 ** -133                                  # subnormal of bf16
    x[0, 32:] = torch.tensor(3.3e38).bfloat16()
    x[1, 0], x[1, 40] = 2.0 ** -126, -2.0 ** 127
    x[2, 5] = float("inf")
    x[3, 40] = float("nan")
    x[4, 7], x[4, 8] = -float("inf"), 1.0
    x[5] = 1.96875                                           # saturates: 504 of 448
    x[6] = torch.linspace(-2, 2, 64).bfloat16()
    out, q, sf = nv.act_checkpoint(x, "relu")
    torch.cuda.synchronize()
    v = ref.f64(x)
    want, s = ref.mxfp8(v)
    codes, _ = untile(sf.cpu().numpy(), 8, 2)
    assert np.array_equal(codes, s) and codes[2, 0] == 255 and codes[3, 1] == 255 and codes[4, 0] == 255
    fine = np.repeat(s != 255, 32, 1)
    assert np.array_equal(e4m3_value(q.cpu().numpy())[fine], want[fine])
    d = torch.ones_like(x)
    dx, act_q, act_sf = nv.act_checkpoint_backward(d, q, sf, "silu", recompute=True)
    torch.cuda.synchronize()
    assert torch.isnan(dx[2, :32]).all() and torch.isnan(dx[3, 32:]).all() and torch.isfinite(dx[2, 32:]).all()
    assert np.isnan(ref.decode(act_q, act_sf, 8, 64)[4, :32]).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n", [(1, 1), (1, 8), (3, 16), (2, 33), (5, 100), (129, 64), (7, 520), (2, 4104), (3, 9000)])
def test_backward(m, n, act):
    k = columns(n, act)
    v = ref.f64(bf16(m, k, m + n))
    q, sf = ref.make_mxfp8(v)
    x = ref.decode(q, sf, m, k)
    dout = bf16(m, n, 5, 0.3, pad=8)
    dx, act_q, act_sf = nv.act_checkpoint_backward(dout, q, sf, act, recompute=True)
    torch.cuda.synchronize()
    want, mag = ref.backward(x, ref.f64(dout), act)
    assert np.all(np.abs(ref.f64(dx) - want) <= HALF * np.abs(want) + EPS * mag + tiny(x, ref.f64(dout)))
    # the activation's codes: those of a value within EPS
    f = ref.forward(x, act)
    vals, s = ref.mxfp8(f)
    kp = (n + 31) // 32 * 32
    codes, full = untile(act_sf.cpu().numpy(), m, kp // 32)
    amax = np.abs(np.pad(f, ((0, 0), (0, kp - n))).reshape(m, -1, 32)).max(2)
    _, frac = np.divmod(np.log2(np.where(amax > 0, amax, 1.0)), 1.0)
    sure = np.minimum(frac, 1 - frac) > 2 * EPS
    assert np.array_equal(codes[sure], s[sure])
    got = ref.decode(act_q, act_sf, m, n)
    scale = np.repeat(2.0 ** (codes - 127.0), 32, 1)[:, :n]
    # half an E4M3 step, 2^-4 of the value or 2^-10 below 2^-6; values past 448 saturate
    bound = np.maximum(np.maximum(2.0 ** -4 * np.abs(f), 2.0 ** -10 * scale), np.abs(f) - 448 * scale)
    assert np.all(np.abs(got - f) <= bound + EPS * np.abs(f) + tiny(x))
    # a rounding moves for values within EPS of a threshold, EPS / 2^-4 * 2 of them: 2^-10
    same = (got == (vals.reshape(m, -1, 32) * 2.0 ** (s - 127.0)[..., None]).reshape(m, -1)[:, :n]).mean()
    assert same >= 1 - 2.0 ** -10 - 2.0 / got.size
    pad = full.copy()
    pad[:m, :kp // 32] = 0
    assert not pad.any()
    assert (act_q.cpu().numpy()[:, n:] & 127 == 0).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "swiglu", "geglu"])
def test_gradient_against_differences(act):
    """Central differences in 64 bits: off by h^2 / 6 of a third derivative below 4 (and the kernel as above)."""
    n, h = 32, 2.0 ** -12
    k = columns(n, act)
    q, sf = ref.make_mxfp8(ref.f64(bf16(4, k, 3)) + 0.01)
    x = ref.decode(q, sf, 4, k)
    dout = bf16(4, n, 4)
    d = ref.f64(dout)
    got = ref.f64(nv.act_checkpoint_backward(dout, q, sf, act)[0])
    _, mag = ref.backward(x, d, act)
    for c in range(k):
        step = np.zeros_like(x)
        step[:, c] = h * np.maximum(1.0, np.abs(x[:, c]))
        diff = ((ref.forward(x + step, act) - ref.forward(x - step, act)) * d).sum(1) / (2 * step[:, c])
        other = np.abs(x[:, c ^ 1]) if k == 2 * n else 1.0
        tol = HALF * np.abs(diff) + EPS * mag[:, c] + 16 * h * h * np.abs(d[:, c // 2 if k == 2 * n else c]) * np.maximum(other, 1) * np.maximum(1, x[:, c] ** 2)
        kink = (act == "relu") & (np.abs(x[:, c]) <= 2 * step[:, c])
        assert np.all((np.abs(got[:, c] - diff) <= tol) | kink), c


def test_either_half_of_the_backward_pass():
    """dx alone, the activation alone, and both: the same bits."""
    q, sf = ref.make_mxfp8(ref.f64(bf16(70, 96, 6)))
    dout = bf16(70, 48, 7)
    dx, act_q, act_sf = nv.act_checkpoint_backward(dout, q, sf, "swiglu", recompute=True)
    assert torch.equal(dx, nv.act_checkpoint_backward(dout, q, sf, "swiglu")[0])
    a, s = torch.zeros_like(act_q), torch.zeros_like(act_sf)
    nv.nvfp4_act_checkpoint_backward(None, 0, q, sf, 70, 48, nv.ACTIVATIONS["swiglu"], None, None, 0, None, 0, a, s)
    torch.cuda.synchronize()
    assert torch.equal(a, act_q) and torch.equal(s, act_sf)


def test_large_and_flat_arguments():
    """Where exponentials overflow or vanish: slopes are 0 or 1, nothing is NaN."""
    v = np.array([[1e30, -1e30, 60000.0, -60000.0, 100.0, -100.0, 20.0, -20.0] + [0.0] * 24], np.float64)
    v = np.concatenate([np.pad(v[:, i:i + 1], ((0, 0), (0, 31))) for i in range(8)], 1)
    q, sf = ref.make_mxfp8(v)
    x = ref.decode(q, sf, 1, 256)
    dout = torch.ones(1, 256, dtype=torch.bfloat16, device="cuda")
    for act in ("gelu", "silu", "relu"):
        dx, act_q, act_sf = nv.act_checkpoint_backward(dout, q, sf, act, recompute=True)
        got = ref.f64(dx)
        assert np.isfinite(got).all() and np.isfinite(ref.decode(act_q, act_sf, 1, 256)).all()
        pos = x[0] > 50
        assert np.all(got[0, pos] == 1) and np.all(np.abs(got[0, x[0] < -50]) < 1e-18)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("counts", [[5], [0, 0, 0], [1, 0, 130, 128], [127, 1, 0, 64, 129, 0]])
def test_groups(counts, act):
    """Only the real rows are written; dx's padding rows are zeros; rows behind the last group stay."""
    offsets, cnt, rows, real = ref.groups_of(counts)
    n = 72
    k = columns(n, act)
    x = bf16(rows, k, 8)
    x[torch.from_numpy(~real).cuda()] = float("nan")
    sizes = (rows, nv.padded_k(k)), (nv.nvfp4_mxfp4_scale_bytes(rows, k),)
    q, sf = (torch.full(s, 0x55, dtype=torch.uint8, device="cuda") for s in sizes)
    out = torch.full((rows, n), 3.0, dtype=torch.bfloat16, device="cuda")
    code = nv.ACTIVATIONS[act]
    nv.nvfp4_act_checkpoint(x, x.stride(0), rows, n, code, offsets, cnt, len(counts), out, n, q, sf)
    torch.cuda.synchronize()
    keep = torch.from_numpy(real).cuda()
    dense = nv.act_checkpoint(torch.where(keep[:, None], x, torch.zeros_like(x)), act)
    assert torch.equal(out[keep], dense[0][keep]) and (out[~keep] == 3).all()
    assert torch.equal(q[keep], dense[1][keep]) and (q[~keep] == 0x55).all()
    codes, _ = untile(sf.cpu().numpy(), rows, nv.padded_k(k) // 32)
    dcodes, _ = untile(dense[2].cpu().numpy(), rows, nv.padded_k(k) // 32)
    assert np.array_equal(codes[real], dcodes[real]) and (codes[~real] == 0x55).all()

    dout = bf16(rows, n, 9)
    dout[~keep] = float("nan")
    dx = torch.full((rows, k), 3.0, dtype=torch.bfloat16, device="cuda")
    aq = torch.full((rows, nv.padded_k(n)), 0x55, dtype=torch.uint8, device="cuda")
    asf = torch.full((nv.nvfp4_mxfp4_scale_bytes(rows, n),), 0x55, dtype=torch.uint8, device="cuda")
    nv.nvfp4_act_checkpoint_backward(dout, dout.stride(0), q, sf, rows, n, code, offsets, cnt, len(counts), dx, k, aq, asf)
    torch.cuda.synchronize()
    zero = torch.where(keep[:, None], dout, torch.zeros_like(dout))
    d2 = nv.act_checkpoint_backward(zero, dense[1], dense[2], act, recompute=True)
    last = int(offsets[-1])
    assert torch.equal(dx[keep], d2[0][keep]) and (dx[:last][~keep[:last]] == 0).all() and (dx[last:] == 3).all()
    assert torch.equal(aq[keep], d2[1][keep]) and (aq[~keep] == 0x55).all()


def test_rows_that_end_inside_the_last_groups_padding():
    """A buffer shorter than the groups' padded rows: nothing past it is touched."""
    offsets, cnt, _, _ = ref.groups_of([130, 20])
    rows, n = 256 + 20 + 5, 40                               # the last band has 25 rows
    guard = torch.full((rows + 200, 2 * n), 3.0, dtype=torch.bfloat16, device="cuda")
    x, dout = bf16(rows, 2 * n, 14), bf16(rows, n, 15)
    _, q, sf = nv.act_checkpoint(x, "swiglu", offsets, cnt)
    nv.act_checkpoint_backward(dout, q, sf, "swiglu", offsets, cnt, dx=guard[:rows], recompute=True)
    torch.cuda.synchronize()
    assert (guard[rows:] == 3).all() and (guard[276:rows] == 0).all() and (guard[130:256] == 0).all()
    # counts that claim more rows than there are
    cnt.copy_(torch.tensor([200, 100], device="cuda"))
    guard.fill_(3.0)
    nv.act_checkpoint_backward(dout, q, sf, "swiglu", offsets, cnt, dx=guard[:rows])
    torch.cuda.synchronize()
    assert (guard[rows:] == 3).all()


def test_captured_with_streams():
    """Replays see new data; a second stream's calls do not disturb the first's."""
    x = bf16(300, 256, 10)
    out = torch.zeros(300, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(300, 256, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(nv.nvfp4_mxfp4_scale_bytes(300, 256), dtype=torch.uint8, device="cuda")
    dx, dout = torch.zeros(300, 256, dtype=torch.bfloat16, device="cuda"), bf16(300, 128, 11)

    def step():
        nv.nvfp4_act_checkpoint(x, 256, 300, 128, 4, None, None, 0, out, 128, q, sf)
        nv.nvfp4_act_checkpoint_backward(dout, 128, q, sf, 300, 128, 4, None, None, 0, dx, 256, None, None)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (12, 13):
        x.copy_(bf16(300, 256, seed))
        graph.replay()
        torch.cuda.synchronize()
        want, wq, wsf = nv.act_checkpoint(x, "swiglu")
        assert torch.equal(out, want) and torch.equal(q, wq) and torch.equal(sf, wsf)
        assert torch.equal(dx, nv.act_checkpoint_backward(dout, wq, wsf, "swiglu")[0])
