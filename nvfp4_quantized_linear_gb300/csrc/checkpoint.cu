// 8-bit activation checkpoints: a GEMM's output x goes through its activation and
// is kept in MXFP8 for the backward pass, which reads
//   dx = act'(x) dout   and   act(x) again, in MXFP8, for the next weight gradient.
//
// One pass over memory, so bytes bound it; the arithmetic has to stay below them.  A warp
// takes 512 columns of the rows r, r + 32, r + 64 and r + 96 of a 128-row band: a
// thread 16 columns (half an MX block) of each, so that the four rows' scale codes of 128
// columns are one 16-byte line of the tiled layout.  The forward pass has all four rows'
// loads in flight (8192 x 14336 SWIGLU, 949 MB: 139 us, 6.8 TB/s).  The backward pass
// computes more per byte and takes a row at a time at 40 registers, 48 warps an SM
// (1070 MB: 177 to 186 us, 5.8 to 6.0 TB/s; four rows in flight at 80 registers 205, the
// next rows prefetched behind the arithmetic 249).
#include <algorithm>
#include <climits>

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

// Four E4M3 codes times a factor, as two pairs: neighbours, or with kGated the even ones
// (gates) and the odd ones (ups).
template <bool kGated>
__device__ __forceinline__ void unpack_e4m3x4(uint32_t w, uint64_t factor, uint64_t &a, uint64_t &b)
{
    if constexpr (kGated) w = __byte_perm(w, 0, 0x3120);
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    a = mul2(pack2(f.x, f.y), factor);
    b = mul2(pack2(g.x, g.y), factor);
}

__device__ __forceinline__ uint64_t both(float v) { return pack2(v, v); }

__device__ __forceinline__ float min_nan(float a, float b)
{
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Kinds of activation in the backward pass, gates by their own function.
enum ActKind : int { kSilu, kGelu, kRest };

// The activation and its slope of a pair.  With u = b (v + c v^3) (b = 1, c = 0 for SILU,
// b = 2 sqrt(2 / pi), c = 0.044715 for GELU) both are v sigmoid(u), with slope
// s + v s (1 - s) u'.  The codes of act(v) sit 2^-4 apart, so an error of the value
// shows as a share of codes on the wrong side of a threshold: e = 2^(-u log2 e) has its
// argument split into a whole and a fraction (argument reduction in two steps of fused
// arithmetic, the whole by adding 1.5 * 2^23; one rounding of 2^-25), 1 / (1 + e) a step of
// Newton and Raphson's iteration.  v is clamped where e leaves the floats, beyond which s is 0 or 1 for
// fp32.  (Every minimum and maximum keeps a NaN.)
template <int kKind>
__device__ __forceinline__ void act_and_slope(uint64_t v, bool relu, uint64_t &f, uint64_t &df)
{
    float v0, v1;
    unpack2(v, v0, v1);
    if constexpr (kKind == kRest) {
        f = relu ? pack2(max_nan(v0, 0.0f), max_nan(v1, 0.0f)) : v;
        df = relu ? pack2(v0 > 0.0f ? 1.0f : 0.0f * v0, v1 > 0.0f ? 1.0f : 0.0f * v1) : both(1.0f);
        return;
    }
    constexpr float kLog2e = 1.44269504089f, kB = kKind == kGelu ? 1.5957691216f : 1.0f, kC = 0.044715f;
    constexpr float kLimit = kKind == kGelu ? 9.9f : 87.0f;       // |u| < 87.1 there
    const uint64_t one = both(1.0f), minus = both(-1.0f), magic = both(0x1.8p23f);
    v0 = max_nan(v0, -kLimit);
    v1 = max_nan(v1, -kLimit);
    const uint64_t low = pack2(v0, v1), w = pack2(min_nan(v0, kLimit), min_nan(v1, kLimit));
    uint64_t c = both(-kLog2e * kB), vv = 0;
    if constexpr (kKind == kGelu) {
        vv = mul2(w, w);
        c = fma2(vv, both(-kLog2e * kB * kC), c);
    }
    const uint64_t t = fma2(w, c, magic);                // the whole part in the low bits
    const uint64_t frac = fma2(w, c, fma2(t, minus, magic));
    float t0, t1, x0, x1, e0, e1, r0, r1;
    unpack2(t, t0, t1);
    unpack2(frac, x0, x1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(x0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(x1));
    const uint64_t e = pack2(__int_as_float(__float_as_int(e0) + (__float_as_int(t0) << 23)),
                             __int_as_float(__float_as_int(e1) + (__float_as_int(t1) << 23)));
    const uint64_t d = add2(e, one);
    unpack2(d, x0, x1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(x0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(x1));
    const uint64_t r = pack2(r0, r1);
    const uint64_t s = fma2(mul2(r, minus), fma2(d, r, minus), r);
    f = mul2(low, s);
    const uint64_t bend = mul2(mul2(w, s), mul2(e, s));  // v s (1 - s), 1 - s = e s
    if constexpr (kKind == kGelu) df = fma2(bend, fma2(vv, both(3.0f * kB * kC), both(kB)), s);
    else df = fma2(bend, one, s);
}

// Real rows of a band of the sorted rows of an expert layer: the group that holds it (its
// rows start on a band) and how many of its rows are tokens; padding rows follow.  -1
// behind the last group.  A group per lane, all loads in flight at once.
__device__ __forceinline__ int real_rows(const CheckpointParams &p, int band, int lane)
{
    const int row = band * 128, rows = min(128, max(0, p.m - row));
    if (p.offsets == nullptr) return rows;
    int mine = -1;
#pragma unroll 4
    for (int g = lane; g < p.num_groups; g += 32) {
        const int first = p.offsets[g], end = p.offsets[g + 1], count = p.counts[g];
        if (first <= row && row < end) mine = min(rows, max(0, count - (row - first)));
    }
    return __reduce_max_sync(kFull, mine);
}

// 2 N bf16 (two to a word) from column c on; columns past n are not written.
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t *row, int c, int n, const uint32_t (&w)[N])
{
    uint16_t *o = row + c;
    if (c + 2 * N <= n) {
        if constexpr (N == 8) {
            if ((reinterpret_cast<uintptr_t>(o) & 31) == 0) {
                st_global_v8(o, w);
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            *reinterpret_cast<uint4 *>(o + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 2 * N; ++i)
            if (c + i < n) o[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}

template <int N>
__device__ __forceinline__ void store_bf16(uint16_t *row, int c, int n, const uint64_t (&v)[N])
{
    uint32_t w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = bf16x2_of(v[i]);
    store_bf16(row, c, n, w);
}

// Four fp32 to E4M3 (nearest even, saturating), the first in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// N values of a thread (32 / N lanes a block) into codes; returns the block's scale code.
template <int N>
__device__ __forceinline__ uint32_t store_codes(uint8_t *q, int c, int kp, const uint64_t (&v)[N / 2])
{
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        float a, b;
        unpack2(v[i], a, b);
        amax = max_abs3_nan(amax, a, b);
    }
#pragma unroll
    for (int o = 1; o < 32 / N; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(kFull, amax, o));
    const uint32_t code = mx8_code(amax);
    const float mul = __uint_as_float((254u - min(code, 253u)) << 23);   // 2^-s (a NaN block's codes mean nothing)
    if (c < kp) {
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            float a, b, x, y;
            unpack2(mul2(v[2 * i], both(mul)), a, b);
            unpack2(mul2(v[2 * i + 1], both(mul)), x, y);
            w[i] = e4m3x4(a, b, x, y);
        }
        if constexpr (N == 16) *reinterpret_cast<uint4 *>(q + c) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(q + c) = make_uint2(w[0], w[1]);
    }
    return c < kp ? code : 0;
}

// The four rows' scale codes of a lane's block, row j's in byte j, to the tiled layout: the
// four blocks of 128 columns, kLanes lanes each, trade bytes, and one lane of each block
// stores a row's word.  `rows`: bit j, row j's codes are written.
template <int kLanes>
__device__ __forceinline__ void store_scales(uint8_t *sf, int band, int r, int c, int nbp, uint32_t codes, unsigned rows)
{
    const int lane = threadIdx.x & 31, first = lane & ~(4 * kLanes - 1), j = (lane / kLanes) & 3;
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __shfl_sync(kFull, codes, first + i * kLanes);
    // byte j of each
    const uint32_t lo = __byte_perm(b[0], b[1], j | (4 + j) << 4), hi = __byte_perm(b[2], b[3], j | (4 + j) << 4);
    if (lane % kLanes == 0 && c / 32 < nbp && ((rows >> j) & 1))
        *reinterpret_cast<uint32_t *>(sf + ((int64_t)band * (nbp / 4) + c / 128) * 512 + r * 16 + j * 4) =
            (lo & 0xFFFFu) | (hi << 16);
}

// blockIdx.x = ((band * 4 + quarter of its 32 lines) * split + share of a line's four rows) *
// chunks + chunk; a warp takes its line's share.
struct Place {
    int band, r, c;                                      // the first row's line, the thread's first column
    int j0, j1;                                          // rows r + 32 j, j0 <= j < j1
    __device__ __forceinline__ bool has(int j) const { return j >= j0 && j < j1; }
};

__device__ __forceinline__ Place place_of(int chunks, int split)
{
    const unsigned unit = blockIdx.x / chunks, line = unit / split, share = unit - line * split;
    const int rows = 4 / split;
    return {(int)(line >> 2), (int)(line & 3) * 8 + (int)(threadIdx.x >> 5),
            (int)(blockIdx.x % chunks) * 512 + (int)(threadIdx.x & 31) * 16, (int)share * rows, (int)(share + 1) * rows};
}

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 4) act_checkpoint_kernel(const CheckpointParams p, int chunks, int split)
{
    griddep_launch_dependents();
    griddep_wait();
    const Place at = place_of(chunks, split);
    const int lane = threadIdx.x & 31, c = at.c;
    const int real = real_rows(p, at.band, lane);
    // (without groups the rows past m get zero scales: the last band's padding)
    if (real <= at.r && p.offsets != nullptr) return;
    Raw16 raw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t row = (int64_t)at.band * 128 + at.r + 32 * j;
        raw[j].a = raw[j].b = make_uint4(0, 0, 0, 0);
        if (at.has(j) && at.r + 32 * j < real) raw[j] = load16_coherent(p.x + row * p.ldx, c, p.k);
    }
    const ActParams act = act_params(p.act);
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (!at.has(j) || at.r + 32 * j >= real) continue;       // (the same in the whole warp)
        const int64_t row = (int64_t)at.band * 128 + at.r + 32 * j;
        const uint32_t w[8] = {raw[j].a.x, raw[j].a.y, raw[j].a.z, raw[j].a.w, raw[j].b.x, raw[j].b.y, raw[j].b.z, raw[j].b.w};
        uint64_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bf16x2_to_f32x2(w[i]);
        codes |= store_codes<16>(p.q + row * p.kp, c, p.kp, v) << (8 * j);
        if (p.out != nullptr) {
            uint16_t *out = p.out + row * p.ldo;
            if constexpr (kGated) {
                uint64_t o[4];
                apply_gate(o, v, act);
                store_bf16(out, c / 2, p.n_out, o);
            } else {
                apply_act(v, act);
                store_bf16(out, c, p.n_out, v);
            }
        }
    }
    unsigned rows = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) rows |= (at.has(j) && (p.offsets == nullptr || at.r + 32 * j < real) ? 1u : 0u) << j;
    store_scales<2>(p.sf, at.band, at.r, c, p.nbp, codes, rows);
}

// The gradient and the activation of a warp's line.  kWhole: its 512 columns are all there,
// dx rows are on 32-byte boundaries and both outputs wanted, so that nothing is left to
// check per row (43 instructions an element with the checks; a third of them checks and
// addresses).
template <bool kGated, int kKind, bool kWhole>
__device__ __forceinline__ void backward_line(const CheckpointParams &p, const Place &at, int real)
{
    constexpr int kN = kGated ? 8 : 16;
    const int c = at.c, oc = kGated ? c / 2 : c;         // the first of the activation's columns
    const int64_t row0 = (int64_t)at.band * 128 + at.r;
    uint4 line = make_uint4(0, 0, 0, 0);
    if ((kWhole || c < p.kp) && at.r < real)
        line = ld_global_v4(p.sf + ((int64_t)at.band * (p.nbp / 4) + c / 128) * 512 + at.r * 16);
    const uint8_t *q = p.q + row0 * p.kp + c;
    const uint16_t *dout = p.dout + row0 * p.ldd;
    uint16_t *dx = p.dx + row0 * p.ldg;
    uint8_t *act_q = p.act_q + row0 * p.act_kp;
    const bool relu = p.act == kActRelu, with_dx = kWhole || p.dx != nullptr, with_act = kWhole || p.act_q != nullptr;
    // this lane's block of the four: its byte of each row's word, row j's to byte j
    const uint32_t shift = c / 32 % 4, pick = shift | (4 + shift) << 4;
    const uint32_t scales = (__byte_perm(line.x, line.y, pick) & 0xFFFFu) | __byte_perm(line.z, line.w, pick) << 16;
    uint32_t codes = 0;
    unsigned rows = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j, q += 32 * (int64_t)p.kp, dout += 32 * p.ldd, dx += 32 * p.ldg, act_q += 32 * (int64_t)p.act_kp) {
        if (!at.has(j)) continue;
        if (at.r + 32 * j >= real) {
            if (p.offsets != nullptr && with_dx && row0 + 32 * j < p.m) {    // padding rows of a group
                const uint32_t zero[8] = {};
                if constexpr (kWhole) st_global_v8(dx + c, zero);
                else store_bf16(dx, c, p.k, zero);
            }
            continue;
        }
        rows |= 1u << j;
        uint4 qw = make_uint4(0, 0, 0, 0);
        Raw16 d = {qw, qw};
        if (kWhole || c < p.kp) qw = ld_global_v4(q);
        if constexpr (kWhole) {
            d.a = ld_global_v4(dout + oc);
            if constexpr (!kGated) d.b = ld_global_v4(dout + oc + 8);
        } else if (with_dx) {
            if constexpr (kGated) {
                if (oc < p.n_out) d.a = ld_global_v4(dout + oc);
                if (oc + 8 > p.n_out) d.a = first_of8(d.a, p.n_out - oc);
            } else {
                d = load16_coherent(dout, oc, p.n_out);
            }
        }
        const uint64_t factor = both(e8m0_value((scales >> (8 * j)) & 255));
        const uint32_t w[4] = {qw.x, qw.y, qw.z, qw.w};
        uint64_t o[kN / 2];                              // act(x)
        uint32_t g[8];
        if constexpr (kGated) {
            const uint32_t dw[4] = {d.a.x, d.a.y, d.a.z, d.a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint64_t gate, up, f, df;
                unpack_e4m3x4<true>(w[i], factor, gate, up);
                act_and_slope<kKind>(gate, relu, f, df);
                o[i] = mul2(f, up);
                const uint64_t g2 = bf16x2_to_f32x2(dw[i]);
                float a0, a1, b0, b1;
                unpack2(mul2(mul2(g2, up), df), a0, a1);
                unpack2(mul2(g2, f), b0, b1);
                g[2 * i] = bf16x2_rn(a0, b0);
                g[2 * i + 1] = bf16x2_rn(a1, b1);
            }
        } else {
            const uint32_t dw[8] = {d.a.x, d.a.y, d.a.z, d.a.w, d.b.x, d.b.y, d.b.z, d.b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint64_t v[2], df[2];
                unpack_e4m3x4<false>(w[i], factor, v[0], v[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    act_and_slope<kKind>(v[h], relu, o[2 * i + h], df[h]);
                    g[2 * i + h] = bf16x2_of(mul2(bf16x2_to_f32x2(dw[2 * i + h]), df[h]));
                }
            }
        }
        if constexpr (kWhole) st_global_v8(dx + c, g);
        else if (with_dx) store_bf16(dx, c, p.k, g);
        if (with_act) {
            if (!kWhole && oc + kN > p.n_out) {          // (columns past n_out: zeros, whatever x's padding holds)
#pragma unroll
                for (int i = 0; i < kN / 2; ++i)
                    o[i] = oc + 2 * i >= p.n_out ? 0 : oc + 2 * i + 1 >= p.n_out ? o[i] & 0xFFFFFFFFull : o[i];
            }
            codes |= store_codes<kN>(act_q, oc, kWhole ? INT_MAX : p.act_kp, o) << (8 * j);
        }
    }
    if (p.offsets == nullptr) rows = (1u << at.j1) - (1u << at.j0);   // (zeros for rows past m)
    if (with_act) store_scales<32 / kN>(p.act_sf, at.band, at.r, oc, p.act_nbp, codes, rows);
}

template <bool kGated, int kKind>
__global__ void __launch_bounds__(kThreads, kGated ? 6 : 4) act_checkpoint_backward_kernel(const CheckpointParams p, int chunks, int split)
{
    griddep_launch_dependents();
    griddep_wait();
    const Place at = place_of(chunks, split);
    const int real = real_rows(p, at.band, threadIdx.x & 31);
    if (real < 0) return;
    const int end = (at.c & ~511) + 512;                 // of the warp's columns
    const bool whole = end <= p.k && p.dx != nullptr && p.act_q != nullptr &&
                       (reinterpret_cast<uintptr_t>(p.dx) & 31) == 0 && (p.ldg & 15) == 0;
    if (whole) backward_line<kGated, kKind, true>(p, at, real);
    else backward_line<kGated, kKind, false>(p, at, real);
}

// Four rows a warp, two or one where that leaves an SM fewer than four blocks: a short
// launch is a chain of memory latencies, one for each row of a warp.  Four rows / this
// rule, us: 128 x 14336 SWIGLU 6.2 / 4.6, its gradient 7.1 / 5.9; 333 x 2072 GELU 4.3 / 3.3
// and 6.6 / 5.0; from eight blocks an SM on rows of their own lose (512 routed tokens 9.4
// instead of 7.9, 2048 20 instead of 16).
cudaError_t launch_dependent(void (*kernel)(CheckpointParams, int, int), int64_t columns, int num_sms, cudaStream_t s,
                             const CheckpointParams &p)
{
    const int64_t enough = 4 * (int64_t)num_sms;
    const int chunks = (int)((columns + 511) / 512);
    const int64_t lines = rows_padded(p.m) / 128 * 4 * chunks;
    const int split = lines >= enough ? 1 : lines * 2 >= enough ? 2 : 4;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(lines * split), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, chunks, split);
}

}  // namespace

cudaError_t launch_act_checkpoint(const CheckpointParams &p, int num_sms, cudaStream_t s)
{
    return launch_dependent(act_gated(p.act) ? act_checkpoint_kernel<true> : act_checkpoint_kernel<false>,
                            (int64_t)p.nbp * 32, num_sms, s, p);
}

cudaError_t launch_act_checkpoint_backward(const CheckpointParams &p, int num_sms, cudaStream_t s)
{
    const bool gated = act_gated(p.act);
    // (padding columns of the activation's scales included)
    void (*kernel)(CheckpointParams, int, int) = p.act == kActSwiglu  ? act_checkpoint_backward_kernel<true, kSilu>
                                            : p.act == kActGeglu ? act_checkpoint_backward_kernel<true, kGelu>
                                            : p.act == kActSilu  ? act_checkpoint_backward_kernel<false, kSilu>
                                            : p.act == kActGelu  ? act_checkpoint_backward_kernel<false, kGelu>
                                                                 : act_checkpoint_backward_kernel<false, kRest>;
    return launch_dependent(kernel,
                            std::max<int64_t>((int64_t)p.nbp * 32, (int64_t)p.act_nbp * 32 * (gated ? 2 : 1)),
                            num_sms, s, p);
}

}  // namespace nvfp4
