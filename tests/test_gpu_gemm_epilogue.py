"""GPU tests of the GEMM epilogue (bias, activation, residual) on every path of
the GEMMs and linears, against the 64-bit product of the oracle's quantized
operands followed by the activation in 64 bits.

Tolerance: the output's one rounding to bf16 is at most 2^-8 of the value; the
fp32 accumulation and activation before it are allowed 1e-3 of the output's rms
(they are near 1e-5: exact products, fp32 sums, exp to 2^-20, factors of the
gated product a few rms)."""
import numpy as np
import pytest
import torch

import oracle
from _block_ref import activation, e4m3_value, f64, unpack_fp4
from _helpers import dev_scalar, nv, require_library, syn

pytestmark = pytest.mark.gpu
GATED = ("swiglu", "geglu")
ACTS = ["none", "relu", "gelu", "silu", "swiglu", "geglu"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def decode(packed, sf, mx=False):
    scale = 2.0 ** (sf.astype(np.float64) - 127.0) if mx else e4m3_value(sf)
    return torch.from_numpy(unpack_fp4(packed) * np.repeat(scale, 32 if mx else 16, axis=1)).cuda()


def product(a, b, alpha, bias):
    v = (decode(*a) @ decode(*b).T).cpu().numpy() * alpha
    return v if bias is None else v + f64(bias)


def assert_close(got, ref, what):
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref) - 1.01 * 2.0 ** -8 * np.abs(ref)
    assert err.max() <= 1e-3 * np.sqrt((ref * ref).mean()), f"{what}: {err.max():.3e}"


class Case:
    """Operands of one problem, quantized by the library, with the 64-bit accumulator."""

    def __init__(self, m, k, n, act, bias, res, seed, mx=False, n_extra=0):
        self.m, self.k, self.n, self.act, self.mx = m, k, n, act, mx
        nw = (2 * n if act in GATED else n)
        self.nw = nw + n_extra                                 # weight rows past the ones used
        x = syn.bf16_outlier_channels(m, k, seed)
        w = syn.bf16_normal((self.nw, k), 0.05, seed + 1)
        kx = (k + 7) // 8 * 8
        self.x = torch.full((m, kx), float("nan"), dtype=torch.bfloat16).cuda()
        self.x[:, :k] = x.cuda()
        wd = torch.zeros((self.nw, kx), dtype=torch.bfloat16).cuda()
        wd[:, :k] = w.cuda()
        self.gx, self.gw = syn.global_scale(x), syn.global_scale(w)
        self.gs, self.alpha = dev_scalar(self.gx), dev_scalar(syn.alpha_of(self.gx, self.gw))
        bits_x, bits_w = syn.bf16_bits(x), syn.bf16_bits(w[:nw])
        self.bias = syn.bf16_normal((nw,), 0.5, seed + 2).cuda() if bias else None
        if mx:
            self.w = nv.quant_act_mx(wd[:, :k])
            v = product((*oracle.quantize_mx(bits_x), True), (*oracle.quantize_mx(bits_w), True), 1.0, self.bias)
        else:
            self.w = nv.prepare_weight(wd[:, :k], dev_scalar(self.gw))
            v = product(oracle.quantize(bits_x, self.gx), oracle.quantize(bits_w, self.gw),
                        syn.alpha_of(self.gx, self.gw), self.bias)
        self.ldr = (n + 7) // 8 * 8 + 8
        self.res = None
        self.ref = activation(v, act)
        if res:
            full = syn.bf16_normal((m, self.ldr), 2.0, seed + 3).cuda()
            full[:, n:] = float("nan")
            self.res = full[:, :n]
            self.ref = self.ref + f64(self.res)

    def out(self):
        ldo = (self.n + 7) // 8 * 8 + 16
        self.full = torch.full((self.m + 1, ldo), -7.0, dtype=torch.bfloat16, device="cuda")
        return self.full[:self.m, :self.n]

    def check(self, out, what):
        torch.cuda.synchronize()
        nv.nvfp4_device_error()
        assert (self.full[self.m] == -7.0).all() and (self.full[:, self.n:] == -7.0).all(), "written outside"
        assert_close(f64(out), self.ref, what)

    def linear(self):
        f = nv.mxfp4_linear if self.mx else nv.linear
        args = (self.gs, self.alpha) if not self.mx else ()
        o = f(self.x[:, :self.k], *self.w, self.k, self.n, *args, bias=self.bias, act=self.act, residual=self.res,
              out=self.out())
        self.check(o, "linear")
        return o

    def gemm(self):
        a = nv.ACTIVATIONS[self.act]
        o = self.out()
        x = self.x[:, :self.k]
        if self.mx:
            q = nv.quant_act_mx(x)
            nv.nvfp4_mxfp4_gemm_act(*q, self.m, *self.w, self.nw, self.n, self.k, self.bias, a, self.res, self.ldr, o,
                                    o.stride(0))
        else:
            q = nv.quant_act(x, self.gs)
            nv.nvfp4_gemm_act(*q, self.m, *self.w, self.nw, self.n, self.k, self.alpha, self.bias, a, self.res, self.ldr,
                              o, o.stride(0))
        self.check(o, "gemm")
        return o


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,k,n", [(1, 2048, 520), (16, 512, 264), (37, 1024, 200), (128, 320, 600), (200, 1024, 456)])
def test_linear_every_activation(m, k, n, act):
    """m = 1, 16: the single-launch linear (split K at 2048 columns of K); 37:
    split K; 128: one band; 200: CTA pairs.  Bias and residual throughout."""
    Case(m, k, n, act, True, True, seed=m + n).linear()


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("m", [1, 5, 100, 129, 257])
@pytest.mark.parametrize("n", [1, 77, 130])
def test_odd_columns(m, n, act):
    """Output columns that end anywhere inside a tile, a store chunk or a vector."""
    Case(m, 264, n, act, True, True, seed=7 * m + n).linear()


@pytest.mark.parametrize("act", ["silu", "geglu"])
@pytest.mark.parametrize("bias,res", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("m", [3, 90, 300])
def test_optional_parts(m, bias, res, act):
    c = Case(m, 640, 384, act, bias, res, seed=m)
    c.linear()
    c.gemm()


@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
@pytest.mark.parametrize("m", [2, 64, 140])
def test_mxfp4(m, act):
    c = Case(m, 608, 328, act, True, True, seed=m, mx=True)
    c.linear()
    c.gemm()


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("m,k,n", [(129, 2080, 520), (333, 4104, 328), (640, 2304, 200), (1000, 608, 96)])
def test_few_tiles_over_several_row_bands(m, k, n, act):
    """m > 128 with fewer output tiles than CTA pairs, in both formats."""
    Case(m, k, n, act, True, True, seed=m).linear()
    if act == "gelu":
        Case(m, k, n, act, True, True, seed=m, mx=True).linear()


@pytest.mark.parametrize("act", ["relu", "swiglu"])
def test_weight_rows_past_the_output_are_ignored(act):
    for m in (4, 150):
        Case(m, 512, 100, act, True, False, seed=m, n_extra=156).linear()


def test_many_tiles_per_pair():
    """More tiles than CTA pairs: the staging buffer and its barrier go round."""
    for act in ("gelu", "swiglu"):
        c = Case(2300, 256, 4200 if act == "gelu" else 2100, act, True, True, seed=5)
        c.linear()


@pytest.mark.parametrize("m", [1, 128, 300])
@pytest.mark.parametrize("n", [3, 8, 300, 20005])
def test_plain_gemm_leaves_the_columns_past_n_out_alone(m, n):
    """nvfp4_gemm and nvfp4_linear themselves, any n_out (n = 20005: more tiles
    than SMs, so no split K at m = 128)."""
    c = Case(m, 64, n, "none", True, False, seed=n + m)
    c.linear()
    x_fp4, x_sf = nv.quant_act(c.x[:, :64], c.gs)
    o = c.out()
    nv.nvfp4_gemm(x_fp4, x_sf, m, *c.w, c.nw, n, 64, c.alpha, c.bias, o, o.stride(0))
    c.check(o, "gemm")


@pytest.mark.parametrize("m", [2, 16, 40, 200])
@pytest.mark.parametrize("k", [1, 20, 250, 1027])
def test_columns_of_k_past_the_end_are_not_read(m, k):
    """K not a multiple of 8: the row's padding (NaN) stays out of the product."""
    Case(m, k, 136, "silu", False, False, seed=k + m).linear()
    Case(m, k, 136, "silu", False, False, seed=k + m, mx=True).linear()


def test_none_without_residual_is_the_plain_gemm():
    for m in (1, 60, 400):
        c = Case(m, 1024, 512, "none", True, False, seed=m)
        o = c.gemm()
        q = nv.quant_act(c.x[:, :c.k], c.gs)
        p = torch.empty((m, c.n), dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_gemm(*q, m, *c.w, c.nw, c.n, c.k, c.alpha, c.bias, p, c.n)
        torch.cuda.synchronize()
        assert torch.equal(o.contiguous().view(torch.int16), p.view(torch.int16))


def test_large_arguments_saturate():
    """Activations far outside exp's range: zeros (or the argument), never NaN."""
    m, k, n = 130, 64, 128
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 16] = 6.0, -6.0
    gs = dev_scalar(448.0)
    w = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
    w[0::2, 0], w[1::2, 16] = 3.0e4, 3.0e4                   # columns of +1.8e5 and -1.8e5 times alpha
    w_fp4, w_sf = nv.prepare_weight(w, dev_scalar(448.0 / 3.0e4 * 6 / 6))
    for mm in (3, m):
        for act, neg in (("silu", 0.0), ("gelu", 0.0), ("relu", 0.0)):
            out = torch.empty((mm, n), dtype=torch.bfloat16, device="cuda")
            nv.linear(x[:mm], w_fp4, w_sf, k, n, gs, dev_scalar(1.0), act=act, out=out)
            torch.cuda.synchronize()
            assert torch.isfinite(out).all()
            assert (out[:, 0::2] > 1e3).all() and (out[:, 1::2].abs() == neg).all()


def test_transform_path():
    """The transform quantizer feeds the same epilogue: equal to the GEMM entry
    point on the transform quantizer's own codes, bit for bit."""
    m, k, n, bs = 300, 512, 256, 32
    x = syn.bf16_outlier_channels(m, k, 3).cuda()
    t = syn.random_hadamard_transform(bs, 4).cuda()
    w = syn.bf16_normal((2 * n, k), 0.05, 5).cuda()
    gs, gw = dev_scalar(30.0), syn.global_scale(w)
    w_fp4, w_sf = nv.prepare_weight(w, dev_scalar(gw))
    alpha = dev_scalar(syn.alpha_of(30.0, gw))
    res = syn.bf16_normal((m, n), 1.0, 6).cuda()
    a = nv.linear(x, w_fp4, w_sf, k, n, gs, alpha, transform=t, bs=bs, act="swiglu", residual=res)
    q = nv.quant_act(x, gs, t, bs)
    b = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_gemm_act(*q, m, w_fp4, w_sf, 2 * n, n, k, alpha, None, nv.ACTIVATIONS["swiglu"], res, n, b, n)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("k", [264, 4104])
@pytest.mark.parametrize("act", ["none", "relu", "swiglu"])
def test_grouped(act, k):
    """Each group against its own expert, bias included; bands past the groups
    untouched.  Both shared-memory layouts (short and long K)."""
    group_m, n = [130, 0, 1, 128], 192 if act == "swiglu" else 384
    nw = 384
    offsets = np.concatenate([[0], np.cumsum([(g + 127) // 128 * 128 for g in group_m])]).astype(np.int32)
    rows = int(offsets[-1]) + 128
    x = torch.zeros((rows, k), dtype=torch.bfloat16)
    for g, m in enumerate(group_m):
        x[offsets[g]:offsets[g] + m] = syn.bf16_normal((m, k), 1.0, 50 + g)
    w = syn.bf16_normal((len(group_m) * nw, k), 0.05, 60)
    gx, gw = syn.global_scale(x), syn.global_scale(w)
    bias = syn.bf16_normal((len(group_m) * nw,), 0.5, 61)
    al = syn.alpha_of(gx, gw)
    w_fp4, w_sf = nv.prepare_weight(w.cuda(), dev_scalar(gw))
    a_fp4, a_sf = nv.quant_act(x.cuda(), dev_scalar(gx))
    out = torch.full((rows, n), -5.0, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_grouped_gemm_act(a_fp4, a_sf, rows, torch.from_numpy(offsets).cuda(), len(group_m), w_fp4, w_sf, n, k,
                              torch.full((len(group_m),), al, device="cuda"), bias.cuda(), nv.ACTIVATIONS[act], out, n)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    got = f64(out)
    assert (got[offsets[-1]:] == -5.0).all()
    for g, m in enumerate(group_m):
        if m:
            r = slice(int(offsets[g]), int(offsets[g]) + m)
            v = product(oracle.quantize(syn.bf16_bits(x[r]), gx),
                        oracle.quantize(syn.bf16_bits(w[g * nw:(g + 1) * nw]), gw), al, bias[g * nw:(g + 1) * nw])
            assert_close(got[r], activation(v, act), f"group {g}")


def test_interleave_gate_up():
    g, u = torch.arange(6).view(3, 2), 10 + torch.arange(6).view(3, 2)
    w = nv.interleave_gate_up(g, u)
    assert torch.equal(w[0::2], g) and torch.equal(w[1::2], u)
    assert nv.interleave_gate_up(g[:, 0], u[:, 0]).shape == (6,)
