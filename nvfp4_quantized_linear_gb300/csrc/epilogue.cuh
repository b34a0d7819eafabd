// Activations of the GEMM epilogue: out = bf16(act(alpha * acc + bias) + residual).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace nvfp4 {

// Values of the C ABI's nvfp4_activation.
enum Activation : int32_t {
    kActNone = 0,
    kActRelu = 1,
    kActGelu = 2,       // tanh form
    kActSilu = 3,
    kActSwiglu = 4,     // silu(gate) * up over interleaved columns (gate 2j, up 2j + 1)
    kActGeglu = 5       // gelu(gate) * up
};

__host__ __device__ constexpr bool act_gated(int32_t act) { return act >= kActSwiglu; }

// Epilogue variants of the GEMM kernels: alpha and bias only; an activation; a
// gated activation (half as many output columns).
constexpr int kEpiPlain = 0, kEpiAct = 1, kEpiGated = 2;

// SILU is v * sigmoid(v) and GELU, 0.5 v (1 + tanh u) with u = sqrt(2/pi) (v +
// 0.044715 v^3), is v * sigmoid(2u), which has no cancellation where tanh u is
// near -1.  Both are v / (1 + 2^(v (c1 + c3 v^2))) with coefficients that hold
// -log2(e): one code path with coefficients as data.  SILU's c3 would be 0, which
// makes NaN of an infinite v^2 (|v| > 1.8e19); it is -2^-100, which c1 swallows whole
// below |v| = 2^37 and which has c1's sign above, where 2^x is 0 or infinite anyway.
// (A minimum that keeps v^2 finite instead: 1 to 2 % of a prompt's SWIGLU GEMM.)
// RELU and NONE are max(v, floor) with floor 0 or -inf.  The epilogue's unrolled
// code runs once per tile, so its size counts as much as its instructions: a switch
// over the four functions in every group of eight columns cost 10 us in a launch of
// one tile per CTA (instruction fetches), this form 2 to 4.
struct ActParams {
    float c1, c3;       // SILU, GELU and the gates
    float floor;        // RELU, NONE
    bool sigmoid;
};

__device__ __forceinline__ ActParams act_params(int32_t act)
{
    constexpr float kLog2e = 1.44269504f;
    const bool gelu = act == kActGelu || act == kActGeglu;
    ActParams a;
    a.c1 = gelu ? -2.0f * 0.7978845608f * kLog2e : -kLog2e;
    a.c3 = gelu ? -2.0f * 0.7978845608f * 0.044715f * kLog2e : -0x1p-100f;
    a.floor = act == kActRelu ? 0.0f : __int_as_float(0xff800000);
    a.sigmoid = act != kActRelu && act != kActNone;
    return a;
}

// Two fp32 in one 64-bit register, for the packed FMAs (each half rounds like a
// scalar operation).
__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}

__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two bf16 of a word as two fp32.
__device__ __forceinline__ uint64_t bf16x2_to_f32x2(uint32_t w)
{
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// v / (1 + 2^(v (c1 + c3 v^2))) of a pair: five packed operations and four of
// the special-function unit.  ex2.approx and rcp.approx are good to 2^-22, the
// products to 2^-24 of an exponent below 40 where the result matters: the
// value's error is under 2^-17, against the 2^-9 of its rounding to bf16.
// 2^x = inf gives 0, as does 2^x > 2^126, whose reciprocal is flushed: the value
// itself is under 2^-119 there.
__device__ __forceinline__ uint64_t times_sigmoid2(uint64_t v, const ActParams &a)
{
    float x0, x1, e0, e1, r0, r1;
    unpack2(mul2(v, fma2(mul2(v, v), pack2(a.c3, a.c3), pack2(a.c1, a.c1))), x0, x1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(x0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(x1));
    unpack2(add2(pack2(e0, e1), pack2(1.0f, 1.0f)), e0, e1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(e0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(e1));
    return mul2(v, pack2(r0, r1));
}

// The activation of N pairs.
template <int N>
__device__ __forceinline__ void apply_act(uint64_t (&v)[N], const ActParams &a)
{
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = times_sigmoid2(v[i], a);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x0, x1;
            unpack2(v[i], x0, x1);
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(x0) : "f"(a.floor));
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(x1) : "f"(a.floor));
            v[i] = pack2(x0, x1);
        }
    }
}

// o[i] = {act(gate) * up} of the (gate, up) pairs v[2i], v[2i + 1].
template <int N>
__device__ __forceinline__ void apply_gate(uint64_t (&o)[N], const uint64_t (&v)[2 * N], const ActParams &a)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float g0, u0, g1, u1;
        unpack2(v[2 * i], g0, u0);
        unpack2(v[2 * i + 1], g1, u1);
        o[i] = mul2(times_sigmoid2(pack2(g0, g1), a), pack2(u0, u1));
    }
}

// alpha * acc + bias of eight consecutive columns; s_bias: their biases in shared
// memory, 16-byte aligned (not read without use_bias).
__device__ __forceinline__ void scale_bias8(uint64_t *v, const uint32_t *acc, float alpha, const uint16_t *s_bias,
                                            bool use_bias)
{
    uint4 b = make_uint4(0, 0, 0, 0);
    if (use_bias) b = *reinterpret_cast<const uint4 *>(s_bias);
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
    const uint64_t al = pack2(alpha, alpha);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = fma2(pack2(__uint_as_float(acc[2 * i]), __uint_as_float(acc[2 * i + 1])), al, bf16x2_to_f32x2(w[i]));
}

// o[i] += the i-th of four bf16 pairs packed in `w`.
__device__ __forceinline__ void add_residual8(uint64_t *o, const uint4 &w)
{
    o[0] = add2(o[0], bf16x2_to_f32x2(w.x));
    o[1] = add2(o[1], bf16x2_to_f32x2(w.y));
    o[2] = add2(o[2], bf16x2_to_f32x2(w.z));
    o[3] = add2(o[3], bf16x2_to_f32x2(w.w));
}

__device__ __forceinline__ uint32_t bf16x2_of(uint64_t v)
{
    float lo, hi;
    unpack2(v, lo, hi);
    return bf16x2_rn(lo, hi);
}

__device__ __forceinline__ uint4 bf16x8_of(const uint64_t *o)
{
    return make_uint4(bf16x2_of(o[0]), bf16x2_of(o[1]), bf16x2_of(o[2]), bf16x2_of(o[3]));
}

}  // namespace nvfp4
