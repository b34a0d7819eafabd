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

// Epilogue variants of the GEMM kernels: alpha and bias only, an activation
// and / or a residual, and the gated activations (half as many output columns).
constexpr int kEpiPlain = 0, kEpiAct = 1, kEpiGated = 2;

// v * sigmoid(z), with sigmoid(z) = 1 / (1 + e^-z).  __expf and the fast
// reciprocal are within 2^-20 of the exact value over the range where the
// result is not zero in bf16, whose spacing is 2^-8.  e^-z = inf gives 0.
__device__ __forceinline__ float times_sigmoid(float v, float z) { return v * __fdividef(1.0f, 1.0f + __expf(-z)); }

// gelu(v) = 0.5 v (1 + tanh u) with u = sqrt(2/pi) (v + 0.044715 v^3), written
// as v * sigmoid(2u): no cancellation where tanh u is near -1.
__device__ __forceinline__ float gelu_tanh(float v)
{
    const float z = v * __fmaf_rn(v * v, 2.0f * 0.7978845608f * 0.044715f, 2.0f * 0.7978845608f);
    return times_sigmoid(v, z);
}

__device__ __forceinline__ float apply_act(float v, int32_t act)
{
    if (act == kActRelu) return v < 0.0f ? 0.0f : v;      // (keeps NaN, as fmaxf would not)
    if (act == kActGelu) return gelu_tanh(v);
    if (act == kActSilu) return times_sigmoid(v, v);
    return v;
}

__device__ __forceinline__ float apply_gate(float gate, float up, int32_t act)
{
    return (act == kActGeglu ? gelu_tanh(gate) : times_sigmoid(gate, gate)) * up;
}

}  // namespace nvfp4
