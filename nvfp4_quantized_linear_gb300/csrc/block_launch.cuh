// Parameters and launchers of the operators around the linear layer: the
// quantizing norm (norm_quant.cu) and the mixture-of-experts token movement
// (moe.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace nvfp4 {

// Quantized formats of the norm's output (values of the C ABI's nvfp4_format).
enum Format : int32_t { kFmtNvfp4 = 0, kFmtMxfp4 = 1, kFmtMxfp8 = 2 };

constexpr int64_t kNormMaxK = 65536;     // 1024 threads x 4 steps x 16 elements: a row is one CTA's

struct NormQuantParams {
    const uint16_t *x, *residual, *gamma;   // bf16 bits; residual may be nullptr
    int64_t ldx, ldr, ldh;
    uint16_t *h;                             // [m, ldh] bf16 or nullptr
    float eps;
    float inv_k, inv_k_lo;                   // 1 / k as hi + lo
    int32_t fmt;
    int32_t m, k, kp, nb, nbp, mp;           // as in QuantParams, nb in the format's blocks
    const float *gs;                         // device fp32 (NVFP4)
    uint8_t *q, *sf;
    unsigned int *err_flag;                  // device error word (bounded waits)
};

// Shared memory of an SM that the norm's CTAs may take, what a CTA takes beside
// its ring of rows, and rows of a ring.
constexpr uint32_t kNormRingBytes = 224 * 1024, kNormCtaBytes = 1536;
constexpr int kNormMaxStages = 4;

cudaError_t launch_norm_quant(const NormQuantParams &p, int num_sms, cudaStream_t s);

// Expert counts and top-k the MoE kernels take.
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopk = 64;
constexpr int kMoeSortTile = 1024;           // assignments sorted per step of a block
constexpr int64_t kMoeCombineMaxH = 65535 * 1024;   // column parts of 1024 are the grid's y

struct MoeSortParams {
    const void *ids;                         // int32 or int64 [tokens * topk]
    int32_t id_bytes;
    int32_t n, experts;                      // assignments, experts
    int32_t *offsets, *counts, *dest;
    int32_t *hist;                           // workspace: [blocks][experts]
};

cudaError_t launch_moe_sort(const MoeSortParams &p, int num_sms, cudaStream_t s);

struct MoeRowsParams {
    const uint16_t *x;                       // dispatch: tokens; combine: expert rows
    int64_t ldx;
    const uint16_t *g;                       // combine_backward: gradient of the output
    int64_t ldg;
    const uint16_t *residual;                // combine
    int64_t ldr;
    const float *weights;                    // [tokens, topk] or nullptr
    const int32_t *dest;                     // [tokens, topk]
    int32_t tokens, topk, h, experts, rows;  // rows of the dispatched buffer (x or out)
    const int32_t *offsets, *counts;         // padding rows (dispatch, combine_backward)
    uint16_t *out;
    int64_t ldo;
    float *dw;                               // combine_backward
    // quantizing dispatch
    const float *gs;
    uint8_t *q, *sf;
    int32_t kp, nb, nbp;
};

cudaError_t launch_moe_dispatch(const MoeRowsParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_moe_dispatch_quant(const MoeRowsParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_moe_combine(const MoeRowsParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_moe_combine_backward(const MoeRowsParams &p, int num_sms, cudaStream_t s);

}  // namespace nvfp4
