// C ABI of expert routing, the 8-bit activation checkpoints and the gradients
// (declared and documented in include/nvfp4.h).  Host-side validation and
// launches, as in api.cu.
#include <algorithm>
#include <cmath>

#include "api_util.h"
#include "block_launch.cuh"
#include "common.cuh"
#include "epilogue.cuh"
#include "train_launch.cuh"

using namespace nvfp4::api;

namespace {

// Rows of `cols` elements of `size` bytes.
Range range_rows(const void *p, int64_t rows, int64_t cols, int64_t ld, int size, const char *name)
{
    return range(p, p != nullptr && rows > 0 ? (size_t)((rows - 1) * ld + cols) * size : 0, name);
}

// What routing and its gradient check alike.
nvfp4_status check_route(const void *logits, int type, int64_t ldl, int64_t tokens, int experts, int score, int topk,
                         float scale)
{
    if (type != NVFP4_TYPE_F32 && type != NVFP4_TYPE_BF16) return fail(NVFP4_ERR_INVALID_ARG, "unknown type %d", type);
    if (score != NVFP4_SCORE_SOFTMAX && score != NVFP4_SCORE_SIGMOID)
        return fail(NVFP4_ERR_INVALID_ARG, "unknown score %d", score);
    if (experts < 1 || experts > nvfp4::kMoeMaxExperts)
        return fail(NVFP4_ERR_INVALID_ARG, "experts must be in [1, %d] (got %d)", nvfp4::kMoeMaxExperts, experts);
    if (topk < 1 || topk > nvfp4::kMoeMaxTopk || topk > experts)
        return fail(NVFP4_ERR_INVALID_ARG, "topk must be in [1, min(%d, experts)] (got %d)", nvfp4::kMoeMaxTopk, topk);
    if (tokens < 0 || tokens > kMaxDim / topk)
        return fail(NVFP4_ERR_INVALID_ARG, "tokens out of range: %lld", (long long)tokens);
    if (!std::isfinite(scale)) return fail(NVFP4_ERR_INVALID_ARG, "scale must be finite");
    if (tokens > 0 && logits == nullptr) return fail(NVFP4_ERR_INVALID_ARG, "logits is null");
    if (ldl < experts)
        return fail(NVFP4_ERR_INVALID_ARG, "row stride of logits (%lld) < experts (%d)", (long long)ldl, experts);
    if (reinterpret_cast<uintptr_t>(logits) % (type == NVFP4_TYPE_F32 ? 4 : 2))
        return fail(NVFP4_ERR_ALIGNMENT, "logits must be aligned to their elements");
    return NVFP4_OK;
}

nvfp4_status check_groups(const int32_t *offsets, const int32_t *counts, int num_groups)
{
    if (num_groups < 0 || num_groups > nvfp4::kMoeMaxExperts)
        return fail(NVFP4_ERR_INVALID_ARG, "num_groups must be in [0, %d] (got %d)", nvfp4::kMoeMaxExperts, num_groups);
    if ((offsets != nullptr) != (num_groups > 0) || (counts != nullptr) != (num_groups > 0))
        return fail(NVFP4_ERR_INVALID_ARG, "group_offsets and group_counts go with num_groups > 0, and only with it");
    if (!aligned4(offsets) || !aligned4(counts))
        return fail(NVFP4_ERR_ALIGNMENT, "group_offsets and group_counts must be 4-byte aligned");
    return NVFP4_OK;
}

// An MXFP8 operand of rows x cols: pointers and size.
nvfp4_status check_mxfp8(const uint8_t *q, const uint8_t *sf, int64_t rows, int64_t cols)
{
    if (!q || !sf) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned16(q) || !aligned16(sf)) return fail(NVFP4_ERR_ALIGNMENT, "MXFP8 codes and scales must be 16-byte aligned");
    if (nvfp4::rows_padded(rows) * ((nvfp4::padded_k(cols) + 511) / 512) >= (int64_t(1) << 31))
        return fail(NVFP4_ERR_INVALID_ARG, "tensor too large (%lld x %lld)", (long long)rows, (long long)cols);
    return NVFP4_OK;
}

int32_t mx_cols_padded(int64_t cols) { return (int32_t)((nvfp4::padded_k(cols) / 32 + 3) / 4 * 4); }

// Shapes of the checkpoint calls; *k: columns of x.
nvfp4_status check_act(int64_t m, int64_t n_out, int act, int64_t *k)
{
    if (act < NVFP4_ACT_NONE || act > NVFP4_ACT_GEGLU) return fail(NVFP4_ERR_INVALID_ARG, "unknown activation %d", act);
    if (m < 0 || m > kMaxDim) return fail(NVFP4_ERR_INVALID_ARG, "m out of range: %lld", (long long)m);
    if (n_out < 1 || n_out > kMaxDim / 2) return fail(NVFP4_ERR_INVALID_ARG, "n_out out of range: %lld", (long long)n_out);
    *k = nvfp4::act_gated(act) ? 2 * n_out : n_out;
    return NVFP4_OK;
}

nvfp4::CheckpointParams checkpoint_params(int64_t m, int64_t n_out, int64_t k, int act, const int32_t *offsets,
                                          const int32_t *counts, int num_groups)
{
    nvfp4::CheckpointParams p = {};
    p.m = (int32_t)m;
    p.n_out = (int32_t)n_out;
    p.k = (int32_t)k;
    p.kp = (int32_t)nvfp4::padded_k(k);
    p.nbp = mx_cols_padded(k);
    p.act = act;
    p.offsets = offsets;
    p.counts = counts;
    p.num_groups = num_groups;
    p.act_kp = (int32_t)nvfp4::padded_k(n_out);
    p.act_nbp = mx_cols_padded(n_out);
    return p;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_moe_route(const void *logits, int type, int64_t ldl, const float *bias, int64_t tokens, int experts,
                             int score, int topk, int groups, int group_top, int topk_groups, int renormalize, float scale,
                             int32_t *expert_ids, float *weights, nvfp4_stream_t stream)
{
    nvfp4_status st = check_route(logits, type, ldl, tokens, experts, score, topk, scale);
    if (st != NVFP4_OK) return st;
    if (groups < 1 || groups > nvfp4::kRouteMaxGroups || experts % groups != 0)
        return fail(NVFP4_ERR_INVALID_ARG, "groups must be in [1, %d] and divide experts (got %d)", nvfp4::kRouteMaxGroups,
                    groups);
    if (topk_groups < 1 || topk_groups > groups)
        return fail(NVFP4_ERR_INVALID_ARG, "topk_groups must be in [1, groups] (got %d)", topk_groups);
    if (group_top != 1 && group_top != 2) return fail(NVFP4_ERR_INVALID_ARG, "group_top must be 1 or 2 (got %d)", group_top);
    if (tokens == 0) return ok();
    if (!expert_ids || !weights) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned4(bias) || !aligned4(expert_ids) || !aligned4(weights))
        return fail(NVFP4_ERR_ALIGNMENT, "bias, expert_ids and weights must be 4-byte aligned");
    const size_t n4 = (size_t)(tokens * topk) * 4;
    Range outs[2] = {range(expert_ids, n4, "expert_ids"), range(weights, n4, "weights")};
    Range ins[2] = {range_rows(logits, tokens, experts, ldl, type == NVFP4_TYPE_F32 ? 4 : 2, "logits"),
                    range(bias, bias ? (size_t)experts * 4 : 0, "bias")};
    if ((st = check_aliases(outs, 2, ins, 2)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::RouteParams p = {};
    p.logits = logits;
    p.type = type;
    p.ldl = ldl;
    p.bias = bias;
    p.tokens = (int32_t)tokens;
    p.experts = experts;
    p.score = score;
    p.topk = topk;
    p.groups = groups;
    p.group_top = group_top;
    p.topk_groups = topk_groups;
    p.renorm = renormalize != 0;
    p.scale = scale;
    p.ids = expert_ids;
    p.weights = weights;
    return launch_status(nvfp4::launch_route(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "MoE routing kernel");
}

nvfp4_status nvfp4_moe_route_backward(const float *dweights, const int32_t *expert_ids, const void *logits, int type,
                                      int64_t ldl, int64_t tokens, int experts, int score, int topk, int renormalize,
                                      float scale, void *dlogits, int64_t ldd, nvfp4_stream_t stream)
{
    nvfp4_status st = check_route(logits, type, ldl, tokens, experts, score, topk, scale);
    if (st != NVFP4_OK) return st;
    if (ldd < experts)
        return fail(NVFP4_ERR_INVALID_ARG, "row stride of dlogits (%lld) < experts (%d)", (long long)ldd, experts);
    if (tokens == 0) return ok();
    if (!dweights || !expert_ids || !dlogits) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    const int size = type == NVFP4_TYPE_F32 ? 4 : 2;
    if (!aligned4(dweights) || !aligned4(expert_ids) || reinterpret_cast<uintptr_t>(dlogits) % size)
        return fail(NVFP4_ERR_ALIGNMENT, "dweights, expert_ids and dlogits must be aligned to their elements");
    const size_t n4 = (size_t)(tokens * topk) * 4;
    Range outs[1] = {range_rows(dlogits, tokens, experts, ldd, size, "dlogits")};
    Range ins[3] = {range(dweights, n4, "dweights"), range(expert_ids, n4, "expert_ids"),
                    range_rows(logits, tokens, experts, ldl, size, "logits")};
    if ((st = check_aliases(outs, 1, ins, 3)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::RouteParams p = {};
    p.logits = logits;
    p.type = type;
    p.ldl = ldl;
    p.tokens = (int32_t)tokens;
    p.experts = experts;
    p.score = score;
    p.topk = topk;
    p.renorm = renormalize != 0;
    p.scale = scale;
    p.ids = const_cast<int32_t *>(expert_ids);
    p.dw = dweights;
    p.dlogits = dlogits;
    p.ldd = ldd;
    return launch_status(nvfp4::launch_route_backward(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                         "MoE routing-gradient kernel");
}

nvfp4_status nvfp4_act_checkpoint(const void *x_bf16, int64_t ldx, int64_t m, int64_t n_out, int act,
                                  const int32_t *group_offsets, const int32_t *group_counts, int num_groups,
                                  void *out_bf16, int64_t ldo, uint8_t *q, uint8_t *sf, nvfp4_stream_t stream)
{
    int64_t k = 0;
    nvfp4_status st = check_act(m, n_out, act, &k);
    if (st == NVFP4_OK) st = check_groups(group_offsets, group_counts, num_groups);
    if (st != NVFP4_OK) return st;
    if (m == 0) return ok();
    if ((st = check_rows(x_bf16, k, ldx, "x")) != NVFP4_OK) return st;
    if (out_bf16 != nullptr && (st = check_rows(out_bf16, n_out, ldo, "out")) != NVFP4_OK) return st;
    if ((st = check_mxfp8(q, sf, m, k)) != NVFP4_OK) return st;
    Range outs[3] = {range(q, nvfp4_mxfp8_bytes(m, k), "q"), range(sf, nvfp4_mxfp4_scale_bytes(m, k), "sf"),
                     range2d(out_bf16, m, n_out, ldo, "out")};
    Range ins[3] = {range2d(x_bf16, m, k, ldx, "x"), range(group_offsets, num_groups ? (size_t)(num_groups + 1) * 4 : 0, "group_offsets"),
                    range(group_counts, (size_t)num_groups * 4, "group_counts")};
    if ((st = check_aliases(outs, 3, ins, 3)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::CheckpointParams p = checkpoint_params(m, n_out, k, act, group_offsets, group_counts, num_groups);
    p.x = static_cast<const uint16_t *>(x_bf16);
    p.ldx = ldx;
    p.out = static_cast<uint16_t *>(out_bf16);
    p.ldo = ldo;
    p.q = q;
    p.sf = sf;
    return launch_status(nvfp4::launch_act_checkpoint(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                         "activation-checkpoint kernel");
}

nvfp4_status nvfp4_act_checkpoint_backward(const void *dout_bf16, int64_t ldd, const uint8_t *q, const uint8_t *sf,
                                           int64_t m, int64_t n_out, int act, const int32_t *group_offsets,
                                           const int32_t *group_counts, int num_groups, void *dx_bf16, int64_t ldx,
                                           uint8_t *act_q, uint8_t *act_sf, nvfp4_stream_t stream)
{
    int64_t k = 0;
    nvfp4_status st = check_act(m, n_out, act, &k);
    if (st == NVFP4_OK) st = check_groups(group_offsets, group_counts, num_groups);
    if (st != NVFP4_OK) return st;
    if ((dout_bf16 != nullptr) != (dx_bf16 != nullptr) || (act_q != nullptr) != (act_sf != nullptr))
        return fail(NVFP4_ERR_INVALID_ARG, "dout goes with dx, and act_q with act_sf");
    if (m == 0) return ok();
    if (dx_bf16 == nullptr && act_q == nullptr) return fail(NVFP4_ERR_INVALID_ARG, "no output: dx and act_q are null");
    if (dx_bf16 != nullptr) {
        if ((st = check_rows(dout_bf16, n_out, ldd, "dout")) != NVFP4_OK) return st;
        if ((st = check_rows(dx_bf16, k, ldx, "dx")) != NVFP4_OK) return st;
    }
    if ((st = check_mxfp8(q, sf, m, k)) != NVFP4_OK) return st;
    if (act_q != nullptr && (st = check_mxfp8(act_q, act_sf, m, n_out)) != NVFP4_OK) return st;
    Range outs[3] = {range2d(dx_bf16, m, k, ldx, "dx"),
                     range(act_q, act_q ? nvfp4_mxfp8_bytes(m, n_out) : 0, "act_q"),
                     range(act_sf, act_q ? nvfp4_mxfp4_scale_bytes(m, n_out) : 0, "act_sf")};
    Range ins[5] = {range2d(dout_bf16, m, n_out, ldd, "dout"), range(q, nvfp4_mxfp8_bytes(m, k), "q"),
                    range(sf, nvfp4_mxfp4_scale_bytes(m, k), "sf"),
                    range(group_offsets, num_groups ? (size_t)(num_groups + 1) * 4 : 0, "group_offsets"),
                    range(group_counts, (size_t)num_groups * 4, "group_counts")};
    if ((st = check_aliases(outs, 3, ins, 5)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::CheckpointParams p = checkpoint_params(m, n_out, k, act, group_offsets, group_counts, num_groups);
    p.q = const_cast<uint8_t *>(q);
    p.sf = const_cast<uint8_t *>(sf);
    p.dout = static_cast<const uint16_t *>(dout_bf16);
    p.ldd = ldd;
    p.dx = static_cast<uint16_t *>(dx_bf16);
    p.ldg = ldx;
    p.act_q = act_q;
    p.act_sf = act_sf;
    return launch_status(nvfp4::launch_act_checkpoint_backward(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                         "activation-gradient kernel");
}

size_t nvfp4_checkpoint_wgrad_workspace_bytes(int64_t m, int64_t n, int64_t k, int num_groups)
{
    if (m <= 0 || n <= 0 || k <= 0 || num_groups < 0) return 16;
    return std::max<size_t>(16, nvfp4::wgrad_workspace_bytes(m, n, k, num_groups));
}

nvfp4_status nvfp4_checkpoint_wgrad(const void *dy_bf16, int64_t ldd, const uint8_t *q, const uint8_t *sf, int64_t m,
                                    int64_t n, int64_t k, const int32_t *group_offsets, const int32_t *group_counts,
                                    int num_groups, int type, int accumulate, void *dw, int64_t ldw, void *workspace,
                                    size_t workspace_bytes, nvfp4_stream_t stream)
{
    nvfp4_status st = check_groups(group_offsets, group_counts, num_groups);
    if (st != NVFP4_OK) return st;
    if (type != NVFP4_TYPE_F32 && type != NVFP4_TYPE_BF16) return fail(NVFP4_ERR_INVALID_ARG, "unknown type %d", type);
    if (accumulate && type != NVFP4_TYPE_F32)
        return fail(NVFP4_ERR_INVALID_ARG, "only an fp32 gradient accumulates (bf16 would be rounded at every call)");
    if (m < 0 || m > kMaxDim) return fail(NVFP4_ERR_INVALID_ARG, "m out of range: %lld", (long long)m);
    if (n < 1 || n > kMaxDim) return fail(NVFP4_ERR_INVALID_ARG, "n out of range: %lld", (long long)n);
    if (k < 1 || k > kMaxDim) return fail(NVFP4_ERR_INVALID_ARG, "k out of range: %lld", (long long)k);
    const int64_t weights = std::max(1, num_groups);
    if (weights * ((n + 255) / 256) > kMaxDim / ((k + 255) / 256))
        return fail(NVFP4_ERR_INVALID_ARG, "gradient too large (%lld x %lld x %lld)", (long long)weights, (long long)n, (long long)k);
    if (!dw) return fail(NVFP4_ERR_INVALID_ARG, "dw is null");
    const int size = type == NVFP4_TYPE_F32 ? 4 : 2;
    if (ldw < k) return fail(NVFP4_ERR_INVALID_ARG, "row stride of dw (%lld) < k (%lld)", (long long)ldw, (long long)k);
    if (!aligned16(dw) || ldw * size % 16 != 0)
        return fail(NVFP4_ERR_ALIGNMENT, "dw rows must start on 16-byte boundaries");
    if (m > 0) {
        if ((st = check_rows(dy_bf16, n, ldd, "dy")) != NVFP4_OK) return st;
        if ((st = check_mxfp8(q, sf, m, k)) != NVFP4_OK) return st;
    }
    const size_t need = nvfp4_checkpoint_wgrad_workspace_bytes(m, n, k, num_groups);
    if (!workspace || workspace_bytes < need)
        return fail(NVFP4_ERR_WORKSPACE, "workspace too small: %zu bytes given, %zu needed", workspace ? workspace_bytes : 0,
                    need);
    if (!aligned16(workspace)) return fail(NVFP4_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
    Range outs[2] = {range_rows(dw, weights * n, k, ldw, size, "dw"), range(workspace, need, "workspace")};
    Range ins[5] = {range2d(dy_bf16, m, n, ldd, "dy"), range(q, m > 0 ? nvfp4_mxfp8_bytes(m, k) : 0, "q"),
                    range(sf, m > 0 ? nvfp4_mxfp4_scale_bytes(m, k) : 0, "sf"),
                    range(group_offsets, num_groups ? (size_t)(num_groups + 1) * 4 : 0, "group_offsets"),
                    range(group_counts, (size_t)num_groups * 4, "group_counts")};
    if ((st = check_aliases(outs, 2, ins, 5)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::WgradParams p = {};
    p.m = (int32_t)m;
    p.n = (int32_t)n;
    p.k = (int32_t)k;
    p.kp = (int32_t)nvfp4::padded_k(k);
    p.sf_tiles = mx_cols_padded(k) / 4;
    p.sf = sf;
    p.offsets = group_offsets;
    p.counts = group_counts;
    p.num_groups = (int32_t)weights;
    p.type = type;
    p.accumulate = accumulate != 0;
    p.dw = dw;
    p.ldw = ldw;
    p.wait_ns = nvfp4::kDefaultWaitNs;
    cudaError_t e = nvfp4::device_error_word(&p.err_flag);
    if (e != cudaSuccess) return launch_status(e, "weight-gradient kernel (error word)");
    const char *why = nullptr;
    e = nvfp4::launch_wgrad(p, static_cast<const uint16_t *>(dy_bf16), ldd, q, workspace, num_sms,
                            reinterpret_cast<cudaStream_t>(stream), &why);
    if (why) return fail(NVFP4_ERR_CUDA, "%s", why);
    return launch_status(e, "weight-gradient kernel");
}

}  // extern "C"
