// NVFP4 quantizer core shared by quant_kernel (quant.cu) and the fused
// small-m linear (gemm.cu): the per-block arithmetic and the loads of a block.
// Page "TorchNvFp4LinearKernel" (vLLM PR
// #53319), section 关键源码片段: scaled_fp4_quant with the activation global
// scale, swizzled scales and K padded to the weight's padding.
//
// Per 16-element block (all fp32, round-to-nearest-even, IEEE division):
//   s = (amax * gs) / 6;  sf = e4m3(s);  inv = sf ? gs / e4m3(sf) : 0;
//   q_i = e2m1(v_i * inv)
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"
#include "scale_math.cuh"

namespace nvfp4 {
namespace quant_core {

constexpr unsigned kFull = 0xFFFFFFFFu;

// max(|a|, |b|, |c|): the three-input max.abs.f32 of sm_100 and later (one
// instruction where two two-input maxima with abs operands were needed).
__device__ __forceinline__ float max_abs3(float a, float b, float c)
{
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// MXFP4 scale code of a 32-element block with absolute maximum `amax`:
//     s = clamp(floor(log2 amax) - 2, -127, 127)  (-127 for a zero block),
//     code = s + 127 (UE8M0), and the elements are quantized as e2m1(v * 2^-s).
// floor(log2 amax) comes from the fp32 bits (exponent field, or the top set
// bit of a subnormal).
__device__ __forceinline__ uint32_t mx_scale_code(float amax)
{
    if (amax == 0.0f) return 0;
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23);                       // amax >= 0: no sign bit
    const int fl = e != 0 ? e - 127 : -149 + (31 - __clz((int)u));
    const int s = min(max(fl - 2, -127), 127);
    return (uint32_t)(s + 127);
}

// 2^-s for a scale code (s = code - 127 <= 125 for finite input), built from bits.
__device__ __forceinline__ float mx_scale_mul(uint32_t code) { return __uint_as_float((254u - code) << 23); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Scale code and element multiplier of a block with absolute maximum `amax`:
//   s = (amax * gs) / 6;  sf = e4m3(s);  inv = sf ? gs / e4m3(sf) : 0.
// The division by 6 is div6_rn (scale_math.cuh), which gives the same code sf
// as the IEEE quotient for every input.  gs / e4m3(code) comes from a table of
// the 128 non-negative codes (s >= 0, and satfinite never yields the NaN code)
// that each block fills once with the IEEE division (fill_inv_table).
__device__ __forceinline__ uint32_t block_scale_tab(float amax, float gs, const float *inv_tab, float &inv)
{
    const float s = div6_rn(__fmul_rn(amax, gs));
    const uint32_t sf = cvt_e4m3x2(0.0f, s) & 0x7Fu;
    inv = inv_tab[sf];
    return sf;
}

__device__ __forceinline__ void fill_inv_table(float *inv_tab, float gs)
{
    for (int c = threadIdx.x; c < 128; c += blockDim.x) {
        const float d = e4m3_to_f32((uint32_t)c);
        inv_tab[c] = (d == 0.0f) ? 0.0f : __fdiv_rn(gs, d);
    }
}

// q_i = e2m1(v_i * inv), the products two at a time (mul.rn.f32x2: each lane
// of the pair rounds like a scalar fp32 multiply).
__device__ __forceinline__ uint32_t quant8(const float (&v)[8], float inv)
{
    float q[8];
    uint64_t iv;
    asm("mov.b64 %0, {%1, %1};" : "=l"(iv) : "f"(inv));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        uint64_t a, d;
        asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(v[i]), "f"(v[i + 1]));
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(iv));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(q[i]), "=f"(q[i + 1]) : "l"(d));
    }
    return cvt_e2m1x8(q);
}

// ---------------------------------------------------------------------------
// The 16 elements of a block, as they lie in memory.
struct Raw16 {
    uint4 a, b;
};

// The first n of eight bf16, zeros after them.
__device__ __forceinline__ uint4 first_of8(const uint4 &v, int n)
{
    auto keep = [n](uint32_t w, int i) { return 2 * i + 1 < n ? w : 2 * i < n ? w & 0xFFFFu : 0u; };
    return make_uint4(keep(v.x, 0), keep(v.y, 1), keep(v.z, 2), keep(v.w, 3));
}

// The 16 bf16 at row[k0 ..], zero past k (k0 % 8 == 0, rows on 16 bytes).  The last
// piece of a row is read whole, up to 14 bytes past k inside its aligned 16: element
// by element, a lane at a row's end holds its warp up for a memory latency per
// block (333 x 4104 quantized: 4.2 us instead of 3.8; the norm of 333 x 5128: 4.1
// instead of 3.5).
__device__ __forceinline__ Raw16 load16(const uint16_t *row, int k0, int k, bool row_ok)
{
    Raw16 r;
    r.a = r.b = make_uint4(0, 0, 0, 0);
    if (row_ok && k0 < k) r.a = ld_stream_v4(row + k0);
    if (row_ok && k0 + 8 < k) r.b = ld_stream_v4(row + k0 + 8);
    if (k0 + 16 > k) {
        r.a = first_of8(r.a, k - k0);
        r.b = first_of8(r.b, k - k0 - 8);
    }
    return r;
}

// The same by coherent loads: for kernels that are launched as programmatic
// dependents of the kernel that writes them and so may start before it ends (a
// non-coherent load promises data that is constant from the kernel's start).
__device__ __forceinline__ Raw16 load16_coherent(const uint16_t *row, int k0, int k)
{
    Raw16 r;
    r.a = r.b = make_uint4(0, 0, 0, 0);
    if (k0 < k) r.a = ld_global_v4(row + k0);
    if (k0 + 8 < k) r.b = ld_global_v4(row + k0 + 8);
    if (k0 + 16 > k) {
        r.a = first_of8(r.a, k - k0);
        r.b = first_of8(r.b, k - k0 - 8);
    }
    return r;
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8])
{
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x);
    v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z);
    v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

}  // namespace quant_core
}  // namespace nvfp4
