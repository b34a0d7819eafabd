// Expert routing from router logits, and its gradient.
//
//   l_i  the logit (NaN and -inf: never chosen),  s_i = softmax or sigmoid of l,
//   key_i = s_i + bias_i (l_i without a bias: the scores rise with it),
//   the topk highest keys among the best groups of experts,
//   weight = scale * s, or scale * s / sum of the chosen s.
//
// A warp takes a token; lane i of it owns experts i, i + 32, ... (coalesced rows of
// any alignment).
#include <algorithm>
#include <cfloat>

#include <cuda_bf16.h>

#include "block_launch.cuh"
#include "ptx.cuh"
#include "train_launch.cuh"

namespace nvfp4 {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 4;                                // tokens of a block
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float value_of(float v) { return v; }
__device__ __forceinline__ float value_of(uint16_t bits) { return __uint_as_float((uint32_t)bits << 16); }
__device__ __forceinline__ void store_value(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_value(uint16_t *p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// A logit as the choice sees it: -inf for NaN, +inf as the largest float.
__device__ __forceinline__ float clean(float l) { return l > kNegInf ? fminf(l, FLT_MAX) : kNegInf; }

// Unsigned integers in the order of the floats, 0 for -inf.  (-0 counts as 0.)
__device__ __forceinline__ uint32_t ordered(float f)
{
    const int32_t u = __float_as_int(f + 0.0f);
    return f > kNegInf ? (uint32_t)(u ^ ((u >> 31) | (int32_t)0x80000000)) : 0u;
}

__device__ __forceinline__ uint64_t ordered(double f)
{
    const int64_t u = __double_as_longlong(f + 0.0);
    return f > (double)kNegInf ? (uint64_t)(u ^ ((u >> 63) | (int64_t)0x8000000000000000ll)) : 0ull;
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }

__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// Scores of a row: softmax over its experts (max and sum of exponentials given) or
// sigmoid.
template <typename F>
struct Scores {
    bool softmax;
    F max, sum;
    __device__ __forceinline__ F operator()(F l) const
    {
        return softmax ? exp_of(l - max) / sum : F(1) / (F(1) + exp_of(-l));
    }
};

template <int V, typename F>
__device__ __forceinline__ Scores<F> scores_of(const RouteParams &p, const float (&l)[V])
{
    Scores<F> s = {p.score == kScoreSoftmax, F(0), F(1)};
    if (s.softmax) {
        float m = kNegInf;
#pragma unroll
        for (int v = 0; v < V; ++v) m = fmaxf(m, l[v]);
        m = warp_max(m);
        s.max = m > kNegInf ? F(m) : F(0);
        F sum = F(0);
#pragma unroll
        for (int v = 0; v < V; ++v) sum += exp_of(F(l[v]) - s.max);
        sum = warp_sum(sum);
        s.sum = sum > F(0) ? sum : F(1);
    }
    return s;
}

// Bounds of what the fp32 keys may be off: a score's relative error (expf 2 ulp,
// quotient, sum; for a softmax the rounding of l - max too, at most 2^-24 of the
// distance, which the exponential takes below 2^-25 absolute) and the rounding of
// the sum with the bias.
constexpr float kRelSigmoid = 1.5f * 0x1p-22f, kRelSoftmax = 0x1p-20f, kAbs = 0x1p-24f, kRound = 0x1p-24f;

// The choice with keys of type F: pick[j] = lane + 32 j's expert, -1 for none.
// False if two keys (or groups) whose order matters are too near each other for
// fp32.  s_key: `experts` F of the warp, for groups.
template <int V, typename T, typename F>
__device__ __forceinline__ bool choose(const RouteParams &p, const T *row, const float (&l)[V], F *s_key, int lane,
                                       int (&pick)[2])
{
    const bool by_logit = p.bias == nullptr;
    const bool group_scores = p.groups > 1 && p.group_top == 2;
    Scores<F> score = {false, F(0), F(1)};
    if (!by_logit || group_scores) score = scores_of<V, F>(p, l);
    const float rel = p.score == kScoreSoftmax ? kRelSoftmax : kRelSigmoid;
    F key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        key[v] = F(l[v]);
        const int i = lane + 32 * v;
        if (!by_logit && i < p.experts) {
            const float b = p.bias[i];
            key[v] = l[v] > kNegInf && b > kNegInf ? score(F(l[v])) + F(b) : F(kNegInf);
        }
    }
    bool sure = true;
    if (p.groups > 1) {
        const int size = p.experts / p.groups;
        __syncwarp();
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane + 32 * v < p.experts) s_key[lane + 32 * v] = key[v];
        __syncwarp();
        F top1 = F(kNegInf), top2 = F(kNegInf);
        if (lane < p.groups)
            for (int i = 0; i < size; ++i) {
                const F k = s_key[lane * size + i];
                top2 = k > top1 ? top1 : k > top2 ? k : top2;
                top1 = k > top1 ? k : top1;
            }
        F value = top1;
        if (p.group_top == 2 && top1 > F(kNegInf)) {
            if (by_logit) value = score(top1) + (top2 > F(kNegInf) ? score(top2) : F(0));
            else if (top2 > F(kNegInf)) value = top1 + top2;
        }
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const F other = __shfl_sync(kAll, value, g);
            rank += other > value || (other == value && g < lane) ? 1 : 0;
        }
        const bool kept = lane < p.groups && rank < p.topk_groups;
        const unsigned mask = __ballot_sync(kAll, kept);
        if (sizeof(F) == 4 && (!by_logit || p.group_top == 2)) {
            // the lowest group that stays and the highest that does not
            const float v = (float)value;
            float low = kept ? v : INFINITY, high = lane < p.groups && !kept ? v : kNegInf;
            low = -warp_max(-low);
            high = warp_max(high);
            // (a score is at most 1; two of them and three roundings)
            const float tol = 4.0f * rel + 2.0f * kAbs + 3.0f * kRound * (fabsf(low) + fabsf(high));
            if (high > kNegInf && !(low - high > tol)) sure = false;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (!((mask >> ((lane + 32 * v) / size & 31)) & 1)) key[v] = F(kNegInf);
    }
    using K = decltype(ordered(F(0)));
    K k[V], best = 0;
    int at = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        k[v] = ordered(key[v]);
        if (k[v] > best) { best = k[v]; at = v; }
    }
    const bool check = sizeof(F) == 4 && !by_logit;
    const int rounds = p.topk + (check && p.topk < p.experts ? 1 : 0);
    pick[0] = pick[1] = -1;
    float last = 0.0f, last_l = 0.0f, last_b = 0.0f;
    for (int r = 0; r < rounds; ++r) {
        const K m = warp_max(best);
        if (m == 0) break;
        const int i = (int)__reduce_min_sync(kAll, best == m ? (unsigned)(lane + 32 * at) : kAll);
        const bool mine = lane == (i & 31);
        if (check) {
            // this pick and the one before it; experts of one logit and one bias are
            // equal in any precision (but not the first that is left out: others of
            // its key may be behind it)
            const float b = p.bias[i], li = clean(value_of(row[i]));
            float kf = 0.0f;
            if (mine)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v == at) kf = (float)key[v];
            kf = __shfl_sync(kAll, kf, i & 31);
            if (r > 0) {
                const float s = fmaxf(last - last_b, 0.0f) + fmaxf(kf - b, 0.0f);
                const float tol = rel * s + 2.0f * kAbs + 2.0f * kRound * (fabsf(last) + fabsf(kf));
                const bool same = r < p.topk && li == last_l && b == last_b;
                if (!same && !(last - kf > tol)) sure = false;
            }
            last = kf;
            last_l = li;
            last_b = b;
        }
        if (r < p.topk && lane == (r & 31)) pick[r >> 5] = i;
        if (mine) {
            best = 0;
            const int gone = at;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (v == gone) k[v] = 0;
                if (k[v] > best) { best = k[v]; at = v; }
            }
        }
    }
    return sure;
}

template <int V, typename T>
__global__ void __launch_bounds__(32 * kWarps) moe_route_kernel(const RouteParams p)
{
    extern __shared__ double s_keys[];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= p.tokens) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.ldl;
    float l[V];
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = lane + 32 * v < p.experts ? clean(value_of(row[lane + 32 * v])) : kNegInf;
    int pick[2];
    double *s_key = s_keys + (p.groups > 1 ? warp * p.experts : 0);
    if (!choose<V, T, float>(p, row, l, reinterpret_cast<float *>(s_key), lane, pick))
        choose<V, T, double>(p, row, l, s_key, lane, pick);

    // weights, pick by pick
    float at[2], w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) at[j] = pick[j] >= 0 ? clean(value_of(row[pick[j]])) : kNegInf;
    if (p.renorm) {
        // of the chosen alone, with their largest logit taken out: a softmax over them,
        // or s / e^min(max, 0) for the sigmoid, neither of which underflows in all
        const float top = warp_max(fmaxf(at[0], at[1]));
        const float m = p.score == kScoreSoftmax ? top : fminf(top, 0.0f);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (pick[j] < 0) w[j] = 0.0f;
            else if (p.score == kScoreSoftmax) w[j] = expf(at[j] - m);
            else w[j] = at[j] > 0.0f ? 1.0f / (1.0f + expf(-at[j])) : expf(at[j] - m) / (1.0f + expf(at[j]));
            sum += w[j];
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int j = 0; j < 2; ++j) w[j] = w[j] / sum;
    } else {
        const Scores<float> score = scores_of<V, float>(p, l);
#pragma unroll
        for (int j = 0; j < 2; ++j) w[j] = score(at[j]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (lane + 32 * j < p.topk) {
            p.ids[t * p.topk + lane + 32 * j] = pick[j];
            p.weights[t * p.topk + lane + 32 * j] = pick[j] >= 0 ? p.scale * w[j] : 0.0f;
        }
}

// Gradient.  With g_j = scale * dweights_j of pick j (expert i_j):
//   softmax, renormalised  u = softmax over the picks:  d_j = u_j sum_k u_k (g_j - g_k)
//   sigmoid, renormalised  u = s / sum s:               d_j = (1 - s_j) u_j sum_k u_k (g_j - g_k)
//   sigmoid                d_j = g_j s_j (1 - s_j)
//   softmax                picked:  s_i (G_i * rest + sum_k s_k (G_i - G_k)), others: -s_i sum_k s_k G_k
// where G merges picks of one expert and rest is the sum of the scores of the
// others.  Differences of gradients instead of g_j minus their mean: nothing
// cancels where one pick has nearly all the weight.
template <int V, typename T>
__global__ void __launch_bounds__(32 * kWarps) moe_route_backward_kernel(const RouteParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= p.tokens) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.ldl;
    const bool softmax = p.score == kScoreSoftmax, dense = softmax && !p.renorm;
    int pick[2];
    float at[2], g[2], u[2], d[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int slot = lane + 32 * j;
        const int id = slot < p.topk ? p.ids[t * p.topk + slot] : -1;
        pick[j] = id >= 0 && id < p.experts ? id : -1;
        at[j] = pick[j] >= 0 ? clean(value_of(row[pick[j]])) : kNegInf;
        if (!(at[j] > kNegInf)) pick[j] = -1;
        g[j] = pick[j] >= 0 ? p.scale * p.dw[t * p.topk + slot] : 0.0f;
    }
    float l[V], acc[V], dot = 0.0f;
    if (dense) {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = lane + 32 * v < p.experts ? clean(value_of(row[lane + 32 * v])) : kNegInf;
    }
    if (p.renorm) {
        const float top = warp_max(fmaxf(at[0], at[1]));
        const float m = softmax ? top : fminf(top, 0.0f);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (pick[j] < 0) u[j] = 0.0f;
            else if (softmax) u[j] = expf(at[j] - m);
            else u[j] = at[j] > 0.0f ? 1.0f / (1.0f + expf(-at[j])) : expf(at[j] - m) / (1.0f + expf(at[j]));
            sum += u[j];
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int j = 0; j < 2; ++j) u[j] = pick[j] >= 0 ? u[j] / sum : 0.0f;
    } else if (dense) {
        const Scores<float> score = scores_of<V, float>(p, l);
        // picks of one expert: the first carries their sum
        float merged[2] = {0.0f, 0.0f};
        bool first[2] = {true, true};
        for (int k = 0; k < p.topk; ++k) {
            const int id = __shfl_sync(kAll, pick[k >> 5], k & 31);
            const float gk = __shfl_sync(kAll, g[k >> 5], k & 31);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (id >= 0 && id == pick[j]) {
                    merged[j] += gk;
                    if (k < lane + 32 * j) first[j] = false;
                }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!first[j]) pick[j] = -1;
            g[j] = merged[j];
            u[j] = pick[j] >= 0 ? score(at[j]) : 0.0f;
            dot += u[j] * g[j];
        }
        dot = warp_sum(dot);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = score(l[v]);
        // the others' scores, without those of the picks
        float others = 0.0f;
        unsigned taken = 0;
        for (int k = 0; k < p.topk; ++k) {
            const int id = __shfl_sync(kAll, pick[k >> 5], k & 31);
            if (id >= 0 && (id & 31) == lane) taken |= 1u << (id >> 5);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!((taken >> v) & 1)) others += acc[v];
            acc[v] = (taken >> v) & 1 ? 0.0f : -acc[v] * dot;
        }
        others = warp_sum(others);
#pragma unroll
        for (int j = 0; j < 2; ++j) d[j] = others * g[j];
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            d[j] = pick[j] >= 0 ? g[j] / (1.0f + expf(-at[j])) / (1.0f + expf(at[j])) : 0.0f;
    }
    if (!dense) {
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    }
    if (p.renorm || dense) {
        float sum[2] = {dense ? d[0] : 0.0f, dense ? d[1] : 0.0f};
        for (int k = 0; k < p.topk; ++k) {
            const float uk = __shfl_sync(kAll, u[k >> 5], k & 31);
            const float gk = __shfl_sync(kAll, g[k >> 5], k & 31);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (uk > 0.0f) sum[j] += uk * (g[j] - gk);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            d[j] = pick[j] >= 0 ? u[j] * sum[j] : 0.0f;
            if (p.renorm && !softmax && pick[j] >= 0) d[j] /= 1.0f + expf(at[j]);
        }
    }
    for (int k = 0; k < p.topk; ++k) {
        const int id = __shfl_sync(kAll, pick[k >> 5], k & 31);
        const float dk = __shfl_sync(kAll, d[k >> 5], k & 31);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (id == lane + 32 * v) acc[v] += dk;
    }
    T *out = static_cast<T *>(p.dlogits) + t * p.ldd;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (lane + 32 * v < p.experts) store_value(out + lane + 32 * v, acc[v]);
}

cudaError_t launch_dependent(void (*kernel)(RouteParams), unsigned grid, size_t smem, cudaStream_t s, const RouteParams &p)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

using Kernel = void (*)(RouteParams);

template <typename T>
Kernel route_kernel(int experts)
{
    return experts <= 32    ? moe_route_kernel<1, T>
           : experts <= 64  ? moe_route_kernel<2, T>
           : experts <= 128 ? moe_route_kernel<4, T>
           : experts <= 256 ? moe_route_kernel<8, T>
           : experts <= 512 ? moe_route_kernel<16, T>
                            : moe_route_kernel<32, T>;
}

template <typename T>
Kernel backward_kernel(int experts)
{
    return experts <= 32    ? moe_route_backward_kernel<1, T>
           : experts <= 64  ? moe_route_backward_kernel<2, T>
           : experts <= 128 ? moe_route_backward_kernel<4, T>
           : experts <= 256 ? moe_route_backward_kernel<8, T>
           : experts <= 512 ? moe_route_backward_kernel<16, T>
                            : moe_route_backward_kernel<32, T>;
}

}  // namespace

cudaError_t launch_route(const RouteParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    const Kernel k = p.type == kTypeF32 ? route_kernel<float>(p.experts) : route_kernel<uint16_t>(p.experts);
    const size_t smem = p.groups > 1 ? (size_t)kWarps * p.experts * sizeof(double) : 0;
    return launch_dependent(k, (unsigned)(((int64_t)p.tokens + kWarps - 1) / kWarps), smem, s, p);
}

cudaError_t launch_route_backward(const RouteParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    const Kernel k = p.type == kTypeF32 ? backward_kernel<float>(p.experts) : backward_kernel<uint16_t>(p.experts);
    return launch_dependent(k, (unsigned)(((int64_t)p.tokens + kWarps - 1) / kWarps), 0, s, p);
}

}  // namespace nvfp4
