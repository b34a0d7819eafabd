// C ABI of the operators around the linear layer (declared and documented in
// include/nvfp4.h): the quantizing norm and the mixture-of-experts token
// movement.  Host-side validation and launches, as in api.cu.
#include <algorithm>

#include "api_util.h"
#include "block_launch.cuh"
#include "common.cuh"

using namespace nvfp4::api;

namespace {

// Rows of a dispatched operand: at most min(experts, n) groups, each padded to
// 128 rows.
int64_t moe_rows(int64_t tokens, int topk, int experts)
{
    const int64_t n = tokens * topk;
    return (n + 127 * std::min<int64_t>(experts, n)) / 128 * 128;
}

nvfp4_status check_moe(int64_t tokens, int topk)
{
    if (topk < 1 || topk > nvfp4::kMoeMaxTopk)
        return fail(NVFP4_ERR_INVALID_ARG, "topk must be in [1, %d] (got %d)", nvfp4::kMoeMaxTopk, topk);
    // (a grid of one block per token and 16 per expert stays below 2^31)
    if (tokens < 0 || tokens > (kMaxDim - 16 * nvfp4::kMoeMaxExperts) / topk)
        return fail(NVFP4_ERR_INVALID_ARG, "tokens out of range: %lld", (long long)tokens);
    return NVFP4_OK;
}

nvfp4_status check_experts(int experts)
{
    if (experts < 1 || experts > nvfp4::kMoeMaxExperts)
        return fail(NVFP4_ERR_INVALID_ARG, "experts must be in [1, %d] (got %d)", nvfp4::kMoeMaxExperts, experts);
    return NVFP4_OK;
}

nvfp4_status check_moe_rows(int64_t rows, int64_t h)
{
    if (rows < 0 || rows > kMaxDim) return fail(NVFP4_ERR_INVALID_ARG, "rows out of range: %lld", (long long)rows);
    if (h < 1 || h > kMaxDim) return fail(NVFP4_ERR_INVALID_ARG, "h out of range: %lld", (long long)h);
    return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_add_rmsnorm_quant(const void *x_bf16, int64_t ldx, const void *residual_bf16, int64_t ldr,
                                     const void *gamma_bf16, float eps, int64_t m, int64_t k, int format,
                                     const float *gs_dev, void *h_bf16, int64_t ldh, uint8_t *x_q, uint8_t *x_sf,
                                     nvfp4_stream_t stream)
{
    if (format < NVFP4_FORMAT_NVFP4 || format > NVFP4_FORMAT_MXFP8)
        return fail(NVFP4_ERR_INVALID_ARG, "unknown format %d", format);
    if (m < 0 || m > kMaxDim) return fail(NVFP4_ERR_INVALID_ARG, "m out of range: %lld", (long long)m);
    if (k < 1 || k > nvfp4::kNormMaxK)
        return fail(NVFP4_ERR_INVALID_ARG, "k must be in [1, %lld] (got %lld)", (long long)nvfp4::kNormMaxK, (long long)k);
    if (!(eps >= 0.0f)) return fail(NVFP4_ERR_INVALID_ARG, "eps must be >= 0");
    if (h_bf16 != nullptr && residual_bf16 == nullptr)
        return fail(NVFP4_ERR_INVALID_ARG, "h is the sum with the residual: it needs a residual");
    if (m == 0) return ok();
    nvfp4_status st = check_rows(x_bf16, k, ldx, "x");
    if (st == NVFP4_OK && residual_bf16 != nullptr) st = check_rows(residual_bf16, k, ldr, "residual");
    if (st == NVFP4_OK && h_bf16 != nullptr) st = check_rows(h_bf16, k, ldh, "h");
    if (st != NVFP4_OK) return st;
    const bool nv = format == NVFP4_FORMAT_NVFP4;
    if (!gamma_bf16 || !x_q || !x_sf || (nv && !gs_dev)) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned16(gamma_bf16) || !aligned16(x_q) || !aligned16(x_sf))
        return fail(NVFP4_ERR_ALIGNMENT, "gamma and the quantized outputs must be 16-byte aligned");
    if (nv && !aligned4(gs_dev)) return fail(NVFP4_ERR_ALIGNMENT, "gs must be 4-byte aligned");
    const size_t q_bytes = format == NVFP4_FORMAT_MXFP8 ? nvfp4_mxfp8_bytes(m, k) : nvfp4_packed_bytes(m, k);
    const size_t sf_bytes = nv ? nvfp4_scale_bytes(m, k) : nvfp4_mxfp4_scale_bytes(m, k);
    // h may be x or residual themselves (each thread reads its elements before it writes them)
    const bool in_x = h_bf16 == x_bf16 && ldh == ldx, in_r = h_bf16 == residual_bf16 && ldh == ldr;
    Range outs[3] = {range(x_q, q_bytes, "x_q"), range(x_sf, sf_bytes, "x_sf"), range2d(h_bf16, m, k, ldh, "h")};
    Range ins[4] = {range2d(x_bf16, m, k, ldx, "x"), range2d(residual_bf16, m, k, ldr, "residual"),
                    range(gamma_bf16, (size_t)k * 2, "gamma"), range(gs_dev, nv ? 4 : 0, "gs")};
    if ((st = check_aliases(outs, 2, ins, 4)) != NVFP4_OK) return st;
    Range h_ins[6] = {ins[2], ins[3], outs[0], outs[1]};
    int n_in = 4;
    if (!in_x) h_ins[n_in++] = ins[0];
    if (!in_r) h_ins[n_in++] = ins[1];
    if ((st = check_aliases(outs + 2, 1, h_ins, n_in)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::NormQuantParams p = {};
    p.x = static_cast<const uint16_t *>(x_bf16);
    p.residual = static_cast<const uint16_t *>(residual_bf16);
    p.gamma = static_cast<const uint16_t *>(gamma_bf16);
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldh = ldh;
    p.h = static_cast<uint16_t *>(h_bf16);
    p.eps = eps;
    p.inv_k = (float)(1.0 / (double)k);
    p.inv_k_lo = (float)(1.0 / (double)k - (double)p.inv_k);
    p.fmt = format;
    p.m = (int32_t)m;
    p.k = (int32_t)k;
    p.kp = (int32_t)nvfp4::padded_k(k);
    p.nb = p.kp / (nv ? 16 : 32);
    p.nbp = (p.nb + 3) / 4 * 4;
    p.mp = (int32_t)nvfp4::rows_padded(m);
    p.gs = gs_dev;
    p.q = x_q;
    p.sf = x_sf;
    return launch_status(nvfp4::launch_norm_quant(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                         "norm-quantize kernel");
}

size_t nvfp4_mxfp8_bytes(int64_t rows, int64_t k)
{
    if (rows <= 0 || k <= 0) return 0;
    return (size_t)rows * (size_t)nvfp4::padded_k(k);
}

int64_t nvfp4_moe_rows(int64_t tokens, int topk, int experts)
{
    if (tokens <= 0 || topk <= 0 || experts <= 0) return 0;
    return moe_rows(tokens, topk, experts);
}

size_t nvfp4_moe_sort_workspace_bytes(int64_t tokens, int topk, int experts)
{
    if (tokens <= 0 || topk <= 0 || experts <= 0) return 16;
    const int64_t tiles = (tokens * topk + nvfp4::kMoeSortTile - 1) / nvfp4::kMoeSortTile;
    return std::max<size_t>(16, (size_t)tiles * (size_t)experts * 4);
}

nvfp4_status nvfp4_moe_sort(const void *expert_ids, int id_bytes, int64_t tokens, int topk, int experts,
                            int32_t *group_offsets, int32_t *group_counts, int32_t *dest, void *workspace,
                            size_t workspace_bytes, nvfp4_stream_t stream)
{
    nvfp4_status st = check_moe(tokens, topk);
    if (st == NVFP4_OK) st = check_experts(experts);
    if (st != NVFP4_OK) return st;
    if (id_bytes != 4 && id_bytes != 8)
        return fail(NVFP4_ERR_INVALID_ARG, "id_bytes must be 4 (int32) or 8 (int64), got %d", id_bytes);
    const int64_t n = tokens * topk;
    if (n + 127 * std::min<int64_t>(experts, n) > kMaxDim)
        return fail(NVFP4_ERR_INVALID_ARG, "too many assignments (%lld)", (long long)n);
    if (!group_offsets || !group_counts || (n > 0 && (!expert_ids || !dest)))
        return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    if (reinterpret_cast<uintptr_t>(expert_ids) % id_bytes || !aligned4(group_offsets) || !aligned4(group_counts) ||
        !aligned4(dest))
        return fail(NVFP4_ERR_ALIGNMENT, "ids, offsets, counts and dest must be aligned to their elements");
    const size_t need = nvfp4_moe_sort_workspace_bytes(tokens, topk, experts);
    if (!workspace || workspace_bytes < need)
        return fail(NVFP4_ERR_WORKSPACE, "workspace too small: %zu bytes given, %zu needed", workspace ? workspace_bytes : 0,
                    need);
    if (!aligned16(workspace)) return fail(NVFP4_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
    Range outs[4] = {range(group_offsets, (size_t)(experts + 1) * 4, "group_offsets"),
                     range(group_counts, (size_t)experts * 4, "group_counts"), range(dest, (size_t)n * 4, "dest"),
                     range(workspace, need, "workspace")};
    Range ins[1] = {range(expert_ids, (size_t)n * id_bytes, "expert_ids")};
    if ((st = check_aliases(outs, 4, ins, 1)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::MoeSortParams p = {};
    p.ids = expert_ids;
    p.id_bytes = id_bytes;
    p.n = (int32_t)n;
    p.experts = experts;
    p.offsets = group_offsets;
    p.counts = group_counts;
    p.dest = dest;
    p.hist = static_cast<int32_t *>(workspace);
    return launch_status(nvfp4::launch_moe_sort(p, num_sms, reinterpret_cast<cudaStream_t>(stream)), "MoE sort kernel");
}

nvfp4_status nvfp4_moe_dispatch(const void *x_bf16, int64_t ldx, const int32_t *dest, int64_t tokens, int topk,
                                int64_t rows, int64_t h, const int32_t *group_offsets, const int32_t *group_counts,
                                int experts, void *out_bf16, int64_t ldo, nvfp4_stream_t stream)
{
    nvfp4_status st = check_moe(tokens, topk);
    if (st == NVFP4_OK) st = check_experts(experts);
    if (st == NVFP4_OK) st = check_moe_rows(rows, h);
    if (st != NVFP4_OK) return st;
    if (tokens == 0) return ok();
    if (rows < moe_rows(tokens, topk, experts))
        return fail(NVFP4_ERR_INVALID_ARG, "rows must be at least nvfp4_moe_rows (%lld), got %lld",
                    (long long)moe_rows(tokens, topk, experts), (long long)rows);
    if ((st = check_rows(x_bf16, h, ldx, "x")) != NVFP4_OK) return st;
    if ((st = check_rows(out_bf16, h, ldo, "out")) != NVFP4_OK) return st;
    if (!dest || !group_offsets || !group_counts) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned4(dest) || !aligned4(group_offsets) || !aligned4(group_counts))
        return fail(NVFP4_ERR_ALIGNMENT, "dest, offsets and counts must be 4-byte aligned");
    Range outs[1] = {range2d(out_bf16, rows, h, ldo, "out")};
    Range ins[4] = {range2d(x_bf16, tokens, h, ldx, "x"), range(dest, (size_t)(tokens * topk) * 4, "dest"),
                    range(group_offsets, (size_t)(experts + 1) * 4, "group_offsets"),
                    range(group_counts, (size_t)experts * 4, "group_counts")};
    if ((st = check_aliases(outs, 1, ins, 4)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::MoeRowsParams p = {};
    p.x = static_cast<const uint16_t *>(x_bf16);
    p.ldx = ldx;
    p.dest = dest;
    p.tokens = (int32_t)tokens;
    p.topk = topk;
    p.h = (int32_t)h;
    p.rows = (int32_t)rows;
    p.experts = experts;
    p.offsets = group_offsets;
    p.counts = group_counts;
    p.out = static_cast<uint16_t *>(out_bf16);
    p.ldo = ldo;
    return launch_status(nvfp4::launch_moe_dispatch(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                         "MoE dispatch kernel");
}

nvfp4_status nvfp4_moe_dispatch_quant(const void *x_bf16, int64_t ldx, const float *gs_dev, const int32_t *dest,
                                      int64_t tokens, int topk, int64_t rows, int64_t h, uint8_t *x_fp4,
                                      uint8_t *x_sf, nvfp4_stream_t stream)
{
    nvfp4_status st = check_moe(tokens, topk);
    if (st == NVFP4_OK) st = check_moe_rows(rows, h);
    if (st != NVFP4_OK) return st;
    if (tokens == 0) return ok();
    if (rows < 1) return fail(NVFP4_ERR_INVALID_ARG, "no rows for %lld tokens", (long long)tokens);
    if ((st = check_rows(x_bf16, h, ldx, "x")) != NVFP4_OK) return st;
    if (!gs_dev || !dest || !x_fp4 || !x_sf) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned16(x_fp4) || !aligned16(x_sf))
        return fail(NVFP4_ERR_ALIGNMENT, "packed / scale outputs must be 16-byte aligned");
    if (!aligned4(gs_dev) || !aligned4(dest)) return fail(NVFP4_ERR_ALIGNMENT, "gs and dest must be 4-byte aligned");
    Range outs[2] = {range(x_fp4, nvfp4_packed_bytes(rows, h), "x_fp4"), range(x_sf, nvfp4_scale_bytes(rows, h), "x_sf")};
    Range ins[3] = {range2d(x_bf16, tokens, h, ldx, "x"), range(gs_dev, 4, "gs"),
                    range(dest, (size_t)(tokens * topk) * 4, "dest")};
    if ((st = check_aliases(outs, 2, ins, 3)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::MoeRowsParams p = {};
    p.x = static_cast<const uint16_t *>(x_bf16);
    p.ldx = ldx;
    p.dest = dest;
    p.tokens = (int32_t)tokens;
    p.topk = topk;
    p.h = (int32_t)h;
    p.rows = (int32_t)rows;
    p.gs = gs_dev;
    p.q = x_fp4;
    p.sf = x_sf;
    p.kp = (int32_t)nvfp4::padded_k(h);
    p.nb = p.kp / 16;
    p.nbp = (p.nb + 3) / 4 * 4;
    return launch_status(nvfp4::launch_moe_dispatch_quant(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                         "MoE quantizing dispatch kernel");
}

nvfp4_status nvfp4_moe_combine(const void *y_bf16, int64_t ldy, const float *weights, const int32_t *dest,
                               int64_t tokens, int topk, int64_t rows, int64_t h, const void *residual_bf16,
                               int64_t ldr, void *out_bf16, int64_t ldo, nvfp4_stream_t stream)
{
    nvfp4_status st = check_moe(tokens, topk);
    if (st == NVFP4_OK) st = check_moe_rows(rows, h);
    if (st != NVFP4_OK) return st;
    if (h > nvfp4::kMoeCombineMaxH)
        return fail(NVFP4_ERR_INVALID_ARG, "h must be at most %lld (got %lld)", (long long)nvfp4::kMoeCombineMaxH,
                    (long long)h);
    if (tokens == 0) return ok();
    if (rows < 1) return fail(NVFP4_ERR_INVALID_ARG, "no rows for %lld tokens", (long long)tokens);
    if ((st = check_rows(y_bf16, h, ldy, "y")) != NVFP4_OK) return st;
    if ((st = check_rows(out_bf16, h, ldo, "out")) != NVFP4_OK) return st;
    if (residual_bf16 != nullptr && (st = check_rows(residual_bf16, h, ldr, "residual")) != NVFP4_OK) return st;
    if (!dest) return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned4(dest) || !aligned4(weights))
        return fail(NVFP4_ERR_ALIGNMENT, "weights and dest must be 4-byte aligned");
    Range outs[1] = {range2d(out_bf16, tokens, h, ldo, "out")};
    Range ins[4] = {range2d(y_bf16, rows, h, ldy, "y"),
                    range(weights, weights ? (size_t)(tokens * topk) * 4 : 0, "weights"),
                    range(dest, (size_t)(tokens * topk) * 4, "dest"),
                    range2d(residual_bf16, tokens, h, ldr, "residual")};
    if ((st = check_aliases(outs, 1, ins, 4)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::MoeRowsParams p = {};
    p.x = static_cast<const uint16_t *>(y_bf16);
    p.ldx = ldy;
    p.residual = static_cast<const uint16_t *>(residual_bf16);
    p.ldr = ldr;
    p.weights = weights;
    p.dest = dest;
    p.tokens = (int32_t)tokens;
    p.topk = topk;
    p.h = (int32_t)h;
    p.rows = (int32_t)rows;
    p.out = static_cast<uint16_t *>(out_bf16);
    p.ldo = ldo;
    return launch_status(nvfp4::launch_moe_combine(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                         "MoE combine kernel");
}

nvfp4_status nvfp4_moe_combine_backward(const void *dout_bf16, int64_t ldd, const void *y_bf16, int64_t ldy,
                                        const float *weights, const int32_t *dest, int64_t tokens, int topk,
                                        int64_t rows, int64_t h, const int32_t *group_offsets,
                                        const int32_t *group_counts, int experts, void *dy_bf16, int64_t lddy,
                                        float *dweights, nvfp4_stream_t stream)
{
    nvfp4_status st = check_moe(tokens, topk);
    if (st == NVFP4_OK) st = check_experts(experts);
    if (st == NVFP4_OK) st = check_moe_rows(rows, h);
    if (st != NVFP4_OK) return st;
    if (tokens == 0) return ok();
    if (rows < moe_rows(tokens, topk, experts))
        return fail(NVFP4_ERR_INVALID_ARG, "rows must be at least nvfp4_moe_rows (%lld), got %lld",
                    (long long)moe_rows(tokens, topk, experts), (long long)rows);
    if ((st = check_rows(dout_bf16, h, ldd, "dout")) != NVFP4_OK) return st;
    if ((st = check_rows(y_bf16, h, ldy, "y")) != NVFP4_OK) return st;
    if ((st = check_rows(dy_bf16, h, lddy, "dy")) != NVFP4_OK) return st;
    if (!weights || !dest || !group_offsets || !group_counts || !dweights)
        return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned4(weights) || !aligned4(dest) || !aligned4(group_offsets) || !aligned4(group_counts) ||
        !aligned4(dweights))
        return fail(NVFP4_ERR_ALIGNMENT, "weights, dest, offsets, counts and dweights must be 4-byte aligned");
    const size_t n4 = (size_t)(tokens * topk) * 4;
    Range outs[2] = {range2d(dy_bf16, rows, h, lddy, "dy"), range(dweights, n4, "dweights")};
    Range ins[6] = {range2d(dout_bf16, tokens, h, ldd, "dout"), range2d(y_bf16, rows, h, ldy, "y"),
                    range(weights, n4, "weights"), range(dest, n4, "dest"),
                    range(group_offsets, (size_t)(experts + 1) * 4, "group_offsets"),
                    range(group_counts, (size_t)experts * 4, "group_counts")};
    if ((st = check_aliases(outs, 2, ins, 6)) != NVFP4_OK) return st;
    int num_sms = 0;
    if ((st = current_device(&num_sms)) != NVFP4_OK) return st;
    nvfp4::MoeRowsParams p = {};
    p.x = static_cast<const uint16_t *>(y_bf16);
    p.ldx = ldy;
    p.g = static_cast<const uint16_t *>(dout_bf16);
    p.ldg = ldd;
    p.weights = weights;
    p.dest = dest;
    p.tokens = (int32_t)tokens;
    p.topk = topk;
    p.h = (int32_t)h;
    p.rows = (int32_t)rows;
    p.experts = experts;
    p.offsets = group_offsets;
    p.counts = group_counts;
    p.out = static_cast<uint16_t *>(dy_bf16);
    p.ldo = lddy;
    p.dw = dweights;
    return launch_status(nvfp4::launch_moe_combine_backward(p, num_sms, reinterpret_cast<cudaStream_t>(stream)),
                         "MoE combine-gradient kernel");
}

}  // extern "C"
