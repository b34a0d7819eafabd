// Activations of the GEMM epilogue: out = bf16(act(alpha * acc + bias) + residual).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

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
// -log2(e): one code path with coefficients as data.  RELU and NONE are
// max(v, floor) with floor 0 or -inf.  The epilogue's unrolled code runs once
// per tile, so its size counts as much as its instructions: a switch over the
// four functions in every group of eight columns cost 10 us in a launch of one
// tile per CTA (instruction fetches), this form 2 to 4.
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
    a.c3 = gelu ? -2.0f * 0.7978845608f * 0.044715f * kLog2e : 0.0f;
    a.floor = act == kActRelu ? 0.0f : __int_as_float(0xff800000);
    a.sigmoid = act != kActRelu && act != kActNone;
    return a;
}

// ex2.approx and rcp.approx are good to 2^-22, the products to 2^-24 of an
// exponent below 40 where the result matters: the value's error is under 2^-17,
// against the 2^-9 of its rounding to bf16.  2^x = inf gives 0.
__device__ __forceinline__ float times_sigmoid(float v, const ActParams &a)
{
    const float x = v * __fmaf_rn(v * v, a.c3, a.c1);
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return v * r;
}

template <int N>
__device__ __forceinline__ void apply_act(float (&v)[N], const ActParams &a)
{
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = times_sigmoid(v[i], a);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(v[i]) : "f"(a.floor));
    }
}

// o[i] = act(v[2i]) * v[2i + 1].
template <int N>
__device__ __forceinline__ void apply_gate(float (&o)[N], const float (&v)[2 * N], const ActParams &a)
{
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = times_sigmoid(v[2 * i], a) * v[2 * i + 1];
}

}  // namespace nvfp4
