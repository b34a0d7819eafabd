// 8-bit activation checkpoints: a GEMM's output x goes through its activation and
// is kept in MXFP8 for the backward pass, which reads
//   dx = act'(x) dout   and   act(x) again, in MXFP8, for the next weight gradient.
//
// A thread owns 16 consecutive columns of x, half an MX block; 4 or 2 lanes make a
// block of the activation.  Everything is one pass: bytes bound it.
#include <algorithm>

#include <cuda_bf16.h>

#include "common.cuh"
#include "epilogue.cuh"
#include "ptx.cuh"
#include "quant_core.cuh"
#include "train_launch.cuh"

namespace nvfp4 {
namespace {

using namespace quant_core;

constexpr int kThreads = 256;
constexpr uint32_t kNanCode = 255;                       // E8M0's NaN

// Scale code of an MXFP8 block: s = clamp(floor(log2 amax) - 8, -127, 127), code
// s + 127; the NaN code where an element is not finite.
__device__ __forceinline__ uint32_t mx8_code(float amax)
{
    const int e = (int)(__float_as_uint(amax) >> 23);    // amax >= 0
    return e == 255 ? kNanCode : (uint32_t)max(e - 8, 0);
}

// 2^(code - 127), NaN for the NaN code.
__device__ __forceinline__ float e8m0_value(uint32_t code)
{
    return __uint_as_float(code == kNanCode ? 0x7FC00000u : code == 0 ? 0x00400000u : code << 23);
}

// max(a, |b|, |c|), NaN if one of them is (the plain form drops it).
__device__ __forceinline__ float max_abs3_nan(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ uint32_t e4m3x4(const float *v)
{
    return cvt_e4m3x2(v[1], v[0]) | (cvt_e4m3x2(v[3], v[2]) << 16);
}

// Four E4M3 codes times a factor.
__device__ __forceinline__ void unpack_e4m3x4(uint32_t w, float factor, float *v)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w >> (16 * h))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
        v[2 * h] = f.x * factor;
        v[2 * h + 1] = f.y * factor;
    }
}

// sigmoid(b (v + c v^3)) and its argument's derivative: b = 1, c = 0 for SILU,
// b = 2 sqrt(2 / pi), c = 0.044715 for GELU (v sigmoid(2 u) = 0.5 v (1 + tanh u)).
struct Act {
    float b, bc, bc3;
    bool sigmoid, relu;
};

__device__ __forceinline__ Act act_of(int act)
{
    const bool gelu = act == kActGelu || act == kActGeglu;
    Act a;
    a.b = gelu ? 1.5957691216f : 1.0f;
    a.bc = gelu ? 1.5957691216f * 0.044715f : 0.0f;
    a.bc3 = 3.0f * a.bc;
    a.relu = act == kActRelu;
    a.sigmoid = act != kActRelu && act != kActNone;
    return a;
}

// act(v) and act'(v).
__device__ __forceinline__ void apply(const Act &a, float v, float &f, float &df)
{
    if (a.sigmoid) {
        const float vv = a.bc != 0.0f ? v * v : 0.0f;
        const float u = v * fmaf(a.bc, vv, a.b), du = fmaf(a.bc3, vv, a.b);
        const float e = expf(-fabsf(u));                 // sigmoid and 1 - sigmoid without cancellation
        const float r = 1.0f / (1.0f + e), er = e * r;
        const float s = u >= 0.0f ? r : er, t = u >= 0.0f ? er : r;
        f = v * s;
        df = s == 0.0f || t == 0.0f ? s : fmaf(f * t, du, s);
    } else {
        f = a.relu ? max_nan(v, 0.0f) : v;
        df = a.relu && !(v > 0.0f) ? 0.0f * v : 1.0f;    // (NaN stays NaN)
    }
}

// Whether a row of the sorted rows holds a token (1), is padding of a group (0) or
// lies behind the last group (-1).
__device__ __forceinline__ int row_kind(const CheckpointParams &p, int row)
{
    if (p.offsets == nullptr) return 1;
    int lo = 0, hi = p.num_groups;                       // the last group that starts at or before the row
    if (row >= p.offsets[hi]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.offsets[mid] <= row) lo = mid;
        else hi = mid;
    }
    return row - p.offsets[lo] < p.counts[lo] ? 1 : 0;
}

// 16 (kGated: 8) bf16 from c on; columns past n are not written.
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t *row, int c, int n, const float (&v)[N])
{
    if (c >= n) return;
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = bf16x2_rn(v[2 * i], v[2 * i + 1]);
    if (c + N <= n) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            *reinterpret_cast<uint4 *>(row + c + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i < n) row[c + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}

// N values of a thread (32 / N lanes a block) into codes and the block's scale byte.
template <int N>
__device__ __forceinline__ void store_mxfp8(uint8_t *q, uint8_t *sf, int row, int c, int kp, int nbp, const float (&v)[N])
{
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i += 2) amax = max_abs3_nan(amax, v[i], v[i + 1]);
#pragma unroll
    for (int o = 1; o < 32 / N; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(kFull, amax, o));
    const uint32_t code = mx8_code(amax);
    const float mul = __uint_as_float((254u - min(code, 253u)) << 23);   // 2^-s (a NaN block's codes mean nothing)
    if (c < kp) {
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float u[4] = {v[4 * i] * mul, v[4 * i + 1] * mul, v[4 * i + 2] * mul, v[4 * i + 3] * mul};
            w[i] = e4m3x4(u);
        }
        uint8_t *o = q + (int64_t)row * kp + c;
        if constexpr (N == 16) *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
    }
    if (c % 32 == 0 && c / 32 < nbp) sf[sf_offset(row, c / 32, nbp)] = c < kp ? (uint8_t)code : 0;
}

// Rows and column steps of a block: blockIdx.x = row * steps + step.
template <bool kGated>
__global__ void __launch_bounds__(kThreads) act_checkpoint_kernel(const CheckpointParams p, int steps)
{
    griddep_launch_dependents();
    griddep_wait();
    const int row = blockIdx.x / steps;
    const int c = ((blockIdx.x % steps) * kThreads + threadIdx.x) * 16;
    const int kind = row < p.m ? row_kind(p, row) : 0;
    if (row >= p.m ? p.offsets != nullptr : kind <= 0) return;
    if (row >= p.m) {                                    // padding rows of the last scale band
        if (c % 32 == 0 && c / 32 < p.nbp) p.sf[sf_offset(row, c / 32, p.nbp)] = 0;
        return;
    }
    const Raw16 raw = load16_coherent(p.x + (int64_t)row * p.ldx, c, p.k);
    float v[16];
    unpack8(raw.a, *reinterpret_cast<float(*)[8]>(v));
    unpack8(raw.b, *reinterpret_cast<float(*)[8]>(v + 8));
    if (p.out != nullptr) {
        const Act act = act_of(p.act);
        uint16_t *out = p.out + (int64_t)row * p.ldo;
        float f[kGated ? 8 : 16], df;
#pragma unroll
        for (int i = 0; i < (kGated ? 8 : 16); ++i) {
            apply(act, v[kGated ? 2 * i : i], f[i], df);
            if (kGated) f[i] *= v[2 * i + 1];
        }
        store_bf16(out, kGated ? c / 2 : c, p.n_out, f);
    }
    store_mxfp8(p.q, p.sf, row, c, p.kp, p.nbp, v);
}

template <bool kGated>
__global__ void __launch_bounds__(kThreads) act_checkpoint_backward_kernel(const CheckpointParams p, int steps)
{
    griddep_launch_dependents();
    griddep_wait();
    const int row = blockIdx.x / steps;
    const int c = ((blockIdx.x % steps) * kThreads + threadIdx.x) * 16;
    constexpr int kN = kGated ? 8 : 16;
    const int oc = kGated ? c / 2 : c;                   // the first of the activation's columns
    const int kind = row < p.m ? row_kind(p, row) : -1;
    if (row >= p.m) {
        if (p.offsets == nullptr && p.act_q != nullptr && oc % 32 == 0 && oc / 32 < p.act_nbp)
            p.act_sf[sf_offset(row, oc / 32, p.act_nbp)] = 0;
        return;
    }
    if (kind < 0) return;
    if (kind == 0) {
        const float zero[16] = {};
        if (p.dx != nullptr) store_bf16(p.dx + (int64_t)row * p.ldg, c, p.k, zero);
        return;
    }
    uint4 w = make_uint4(0, 0, 0, 0);
    float factor = 0.0f;
    if (c < p.kp) {
        w = ld_global_v4(p.q + (int64_t)row * p.kp + c);
        factor = e8m0_value(p.sf[sf_offset(row, c / 32, p.nbp)]);
    }
    float v[16];
    unpack_e4m3x4(w.x, factor, v);
    unpack_e4m3x4(w.y, factor, v + 4);
    unpack_e4m3x4(w.z, factor, v + 8);
    unpack_e4m3x4(w.w, factor, v + 12);
    float d[16] = {};
    if (p.dx != nullptr) {
        const uint16_t *dout = p.dout + (int64_t)row * p.ldd;
        if constexpr (kGated) {
            uint4 r = make_uint4(0, 0, 0, 0);
            if (oc < p.n_out) r = first_of8(ld_global_v4(dout + oc), p.n_out - oc);
            unpack8(r, *reinterpret_cast<float(*)[8]>(d));
        } else {
            const Raw16 r = load16_coherent(dout, oc, p.n_out);
            unpack8(r.a, *reinterpret_cast<float(*)[8]>(d));
            unpack8(r.b, *reinterpret_cast<float(*)[8]>(d + 8));
        }
    }
    const Act act = act_of(p.act);
    float f[kN], g[16];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        float df;
        if constexpr (kGated) {
            apply(act, v[2 * i], f[i], df);
            g[2 * i] = d[i] * v[2 * i + 1] * df;
            g[2 * i + 1] = d[i] * f[i];
            f[i] *= v[2 * i + 1];
        } else {
            apply(act, v[i], f[i], df);
            g[i] = d[i] * df;
        }
    }
    if (p.dx != nullptr) store_bf16(p.dx + (int64_t)row * p.ldg, c, p.k, g);
    if (p.act_q != nullptr) {
        if (oc >= p.n_out)                               // (columns past n_out: zeros, whatever x's padding holds)
#pragma unroll
            for (int i = 0; i < kN; ++i) f[i] = 0.0f;
        store_mxfp8(p.act_q, p.act_sf, row, oc, p.act_kp, p.act_nbp, f);
    }
}

cudaError_t launch_dependent(void (*kernel)(CheckpointParams, int), unsigned grid, cudaStream_t s, const CheckpointParams &p,
                             int steps)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, steps);
}

// Column steps of a row (padding columns of the scales included).
int steps_of(int64_t columns) { return (int)((columns + 16 * kThreads - 1) / (16 * kThreads)); }

}  // namespace

cudaError_t launch_act_checkpoint(const CheckpointParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    const int steps = steps_of((int64_t)p.nbp * 32);
    const int64_t rows = p.offsets != nullptr ? p.m : rows_padded(p.m);
    return launch_dependent(act_gated(p.act) ? act_checkpoint_kernel<true> : act_checkpoint_kernel<false>,
                            (unsigned)(rows * steps), s, p, steps);
}

cudaError_t launch_act_checkpoint_backward(const CheckpointParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    const int per = act_gated(p.act) ? 2 : 1;
    const int steps = steps_of(std::max<int64_t>((int64_t)p.nbp * 32, (int64_t)p.act_nbp * 32 * per));
    const int64_t rows = p.offsets != nullptr ? p.m : rows_padded(p.m);
    return launch_dependent(per == 2 ? act_checkpoint_backward_kernel<true> : act_checkpoint_backward_kernel<false>,
                            (unsigned)(rows * steps), s, p, steps);
}

}  // namespace nvfp4
