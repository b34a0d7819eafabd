// Parameters and launchers of expert routing (route.cu), the 8-bit activation
// checkpoints (checkpoint.cu) and the weight gradient from them (wgrad.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace nvfp4 {

enum Score : int32_t { kScoreSoftmax = 0, kScoreSigmoid = 1 };
enum Type : int32_t { kTypeF32 = 0, kTypeBf16 = 1 };

constexpr int kRouteMaxGroups = 32;          // a group per lane

struct RouteParams {
    const void *logits;                      // [tokens, ldl] of `type`
    int32_t type;
    int64_t ldl;
    const float *bias;                       // [experts] or nullptr (forward)
    int32_t tokens, experts, score, topk;
    int32_t groups, group_top, topk_groups;
    int32_t renorm;
    float scale;
    int32_t *ids;                            // [tokens, topk] (backward: read only)
    float *weights;                          // [tokens, topk]
    const float *dw;                         // backward
    void *dlogits;
    int64_t ldd;
};

cudaError_t launch_route(const RouteParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_route_backward(const RouteParams &p, int num_sms, cudaStream_t s);

struct CheckpointParams {
    int32_t m, n_out, k, kp, nbp;            // x: k columns, padded, scale columns padded to 4
    int32_t act;
    const int32_t *offsets, *counts;         // groups' rows, or nullptr
    int32_t num_groups;
    const uint16_t *x;                       // forward
    int64_t ldx;
    uint16_t *out;                           // forward, may be nullptr
    int64_t ldo;
    uint8_t *q, *sf;                         // (backward: read only)
    const uint16_t *dout;                    // backward
    int64_t ldd;
    uint16_t *dx;                            // nullptr: no gradient
    int64_t ldg;
    uint8_t *act_q, *act_sf;                 // nullptr: no activation
    int32_t act_kp, act_nbp;
};

cudaError_t launch_act_checkpoint(const CheckpointParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_act_checkpoint_backward(const CheckpointParams &p, int num_sms, cudaStream_t s);

struct WgradParams {
    int32_t m, n, k, kp;
    int32_t sf_tiles;                        // 512-byte scale tiles per 128-row band
    const uint8_t *sf;
    const int32_t *offsets, *counts;         // groups' rows, or nullptr
    int32_t num_groups;                      // >= 1; without groups row ranges of `span` rows
    int32_t span;
    int32_t part_rows;                       // rows of one accumulator
    int32_t type, accumulate;
    void *dw;                                // [num_groups][n][ldw], dw_cols columns
    int64_t ldw;
    int32_t dw_cols;
    int32_t num_n_blk, num_k_blk;
    unsigned int *err_flag;                  // device error word (bounded waits)
    uint64_t wait_ns;
};

cudaError_t launch_wgrad(const WgradParams &p, const uint16_t *dy, int64_t ldd, const uint8_t *q, void *workspace,
                         int num_sms, cudaStream_t s, const char **why);
size_t wgrad_workspace_bytes(int64_t m, int64_t n, int64_t k, int groups);

}  // namespace nvfp4
