// Expert routing from router logits, and its gradient.
//
//   l_i  the logit (NaN and -inf: never chosen),  s_i = softmax or sigmoid of l,
//   key_i = s_i + bias_i (l_i without a bias: the scores rise with it),
//   the topk highest keys among the best groups of experts,
//   weight = scale * s, or scale * s / sum of the chosen s.
//
// A warp takes a token; its logits are read once.  The bytes are few (16384 tokens of 128
// bf16 logits: 0.8 us), the instructions of picking the experts one by one bound it: 270
// a token there (5.6 us), 1010 with sigmoid scores, a bias and 8 groups of 256 experts (4099
// tokens: 7.7 us), where most of them are scores and groups.  A pick is one maximum over
// the warp of words that hold key and expert; a first form, two maxima a pick over unsorted
// fp32 keys, took 15.4 and 26 us.
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

// V values side by side (aligned as load_row's).
template <int V, typename T>
__device__ __forceinline__ void store_vector(T *o, const float (&v)[V])
{
    constexpr int kBytes = V * (int)sizeof(T), kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (V >= 2) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = bf16x2_rn(v[2 * i], v[2 * i + 1]);
    } else {
        w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
    if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            reinterpret_cast<uint4 *>(o)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
    } else if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t *>(o) = w[0];
    } else {
        *reinterpret_cast<uint16_t *>(o) = (uint16_t)w[0];
    }
}

// A logit as the choice sees it: -inf for NaN, +inf as the largest float.
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, kNegInf), FLT_MAX); }   // (fmaxf drops a NaN)

// Unsigned integers in the order of the floats, 0 for -inf.  (-0 counts as 0.)
__device__ __forceinline__ uint32_t ordered(float f)
{
    const int32_t u = __float_as_int(f + 0.0f);
    return f > kNegInf ? (uint32_t)(u ^ ((u >> 31) | (int32_t)0x80000000)) : 0u;
}

__device__ __forceinline__ float unordered(uint32_t o)
{
    return o == 0u ? kNegInf : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ uint64_t ordered(double f)
{
    const int64_t u = __double_as_longlong(f + 0.0);
    return f > (double)kNegInf ? (uint64_t)(u ^ ((u >> 63) | (int64_t)0x8000000000000000ll)) : 0ull;
}

__device__ __forceinline__ double unordered(uint64_t o)
{
    return __longlong_as_double((int64_t)(o >> 63 ? o ^ 0x8000000000000000ull : ~o));
}

__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(kAll, ordered(v))); }

template <typename F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Good to 1 ulp; 0 from 2^126 on.
__device__ __forceinline__ float reciprocal(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Scores of a row: softmax over its experts (max and sum of exponentials given) or
// sigmoid.  (__fdividef: good to 2 ulp below 2^126.)
struct Scores {
    bool softmax;
    float max, sum;
    __device__ __forceinline__ float operator()(float l) const
    {
        return softmax ? __fdividef(expf(l - max), sum) : reciprocal(1.0f + expf(-l));
    }
};

template <int V>
__device__ __forceinline__ Scores scores_of(const RouteParams &p, const float (&l)[V])
{
    Scores s = {p.score == kScoreSoftmax, 0.0f, 1.0f};
    if (s.softmax) {
        float m = kNegInf;
#pragma unroll
        for (int v = 0; v < V; ++v) m = fmaxf(m, l[v]);
        m = warp_max(m);
        s.max = m > kNegInf ? m : 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += expf(l[v] - s.max);
        sum = warp_sum(sum);
        s.sum = sum > 0.0f ? sum : 1.0f;
    }
    return s;
}

// Bounds of what the fp32 keys may be off, in units of 2^-24 of a score.
//   sigmoid  expf 4 (2 ulp), the sum 1, its reciprocal 2: less than 10
//   softmax  expf 4 and the quotient 4; the sum of V exponentials a lane and of the lanes V + 4,
//            their expf 4; the rounding of l - max, 2^-24 of its distance: in the sum at
//            most the mean distance, below ln(32 V) < 7 (an entropy), in the score itself less
//            than 2^-25 absolute, which kAbs holds: less than V + 24
// Besides the rounding of the sum with the bias.  (Scores below 2^-120 may become 0: far
// below kAbs.)
constexpr float kRelSigmoid = 10 * 0x1p-24f, kAbs = 0x1p-24f, kRound = 0x1p-24f;

template <int V>
__device__ __forceinline__ float relative_error(bool softmax)
{
    return softmax ? (V + 24) * 0x1p-24f : kRelSigmoid;
}

// ------------------------------------------------------------ exact choice ----
// Keys in 64 bits, for the tokens whose order the fast choice below cannot be sure of.  Calls,
// so that their registers and code stay out of the way; p lies in constant memory
// (copied for a call it cost every token 28 stores to local memory).

// The row's keys into s_key (`experts` doubles of the warp): scores with the bias, or the
// logits themselves where nobody asks for scores.  Returns the groups that stay.
template <typename T>
__device__ __noinline__ unsigned exact_keys(const RouteParams &p, const T *row, double *s_key, int lane)
{
    const bool by_logit = p.bias == nullptr, softmax = p.score == kScoreSoftmax;
    const bool scores = !by_logit || (p.groups > 1 && p.group_top == 2);
    const double none = (double)kNegInf;
    double max = none, sum = 1.0;
    if (softmax) {
        float m = kNegInf;
        for (int i = lane; i < p.experts; i += 32) m = fmaxf(m, clean(value_of(row[i])));
        m = warp_max(m);
        max = m > kNegInf ? (double)m : 0.0;
        sum = 0.0;
    }
    __syncwarp();
#pragma unroll 1
    for (int i = lane; i < p.experts; i += 32) {
        const float l = clean(value_of(row[i]));
        double k = (double)l;
        if (scores && l > kNegInf) {
            k = exp(softmax ? k - max : -k);             // (the softmax's quotient follows)
            if (softmax) sum += k;
            else k = 1.0 / (1.0 + k);
        }
        s_key[i] = k;
    }
    if (scores) {
        if (softmax) sum = warp_sum(sum);
        for (int i = lane; i < p.experts; i += 32) {
            const float b = by_logit ? 0.0f : p.bias[i];
            if (s_key[i] > none) s_key[i] = b > kNegInf ? (softmax ? s_key[i] / sum : s_key[i]) + (double)b : none;
        }
    }
    __syncwarp();
    if (p.groups == 1) return ~0u;
    const int size = p.experts / p.groups;
    double top1 = none, top2 = none;
    if (lane < p.groups)
        for (int i = 0; i < size; ++i) {
            const double k = s_key[lane * size + i];
            top2 = k > top1 ? top1 : k > top2 ? k : top2;
            top1 = k > top1 ? k : top1;
        }
    const double value = p.group_top == 2 && top2 > none ? top1 + top2 : top1;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
        const double other = __shfl_sync(kAll, value, g);
        rank += other > value || (other == value && g < lane) ? 1 : 0;
    }
    return __ballot_sync(kAll, lane < p.groups && rank < p.topk_groups);
}

// Of a row's softmax, where a logit is not -inf.
struct ExactSoftmax {
    double max, sum;
};

template <typename T>
__device__ __noinline__ ExactSoftmax exact_softmax(const RouteParams &p, const T *row, int lane)
{
    float m = kNegInf;
    for (int i = lane; i < p.experts; i += 32) m = fmaxf(m, clean(value_of(row[i])));
    const double max = (double)warp_max(m);
    double sum = 0.0;
#pragma unroll 1
    for (int i = lane; i < p.experts; i += 32) sum += exp((double)clean(value_of(row[i])) - max);
    return {max, warp_sum(sum)};
}

// Groups whose values fp32 cannot tell apart: of `kept` those that may be below the best of
// the others, and the others that may be above the lowest of `kept`, are valued again in 64 bits
// (`near`: both; bit g is group g).  Returns the groups that stay.  (Most launches of
// thousands of tokens have such a token and wait for it: 4099 x 256 in 8 groups 7.7 us, with
// every group valued again by exact_keys() 5 more.)
template <typename T>
__device__ __noinline__ unsigned exact_groups(const RouteParams &p, const T *row, unsigned kept, unsigned near, int lane)
{
    const bool softmax = p.score == kScoreSoftmax;
    const int size = p.experts / p.groups;
    ExactSoftmax of = {0.0, 1.0};
    if (softmax) of = exact_softmax(p, row, lane);       // (a group has a value: some logit is not -inf)
    const unsigned sure = kept & ~near;
    double mine = (double)kNegInf;
    for (unsigned left = near; left != 0; left &= left - 1) {
        const int g = __ffs(left) - 1;
        uint64_t best = 0, second = 0;
        for (int i = lane; i < size; i += 32) {
            const int e = g * size + i;
            const float l = clean(value_of(row[e])), b = p.bias != nullptr ? p.bias[e] : 0.0f;
            double k = (double)kNegInf;
            if (l > kNegInf && b > kNegInf) {
                const double x = exp(softmax ? (double)l - of.max : -(double)l);
                k = (softmax ? x / of.sum : 1.0 / (1.0 + x)) + (double)b;
            }
            const uint64_t o = ordered(k);
            second = o > best ? best : o > second ? o : second;
            best = o > best ? o : best;
        }
        const uint64_t first = warp_max(best);
        const int who = __ffs(__ballot_sync(kAll, best == first)) - 1;
        const uint64_t next = warp_max(lane == who ? second : best);
        const double v = unordered(first) + (p.group_top == 2 && next != 0 ? unordered(next) : 0.0);
        if (lane == g && first != 0) mine = v;
    }
    int rank = 0;
    for (unsigned left = near; left != 0; left &= left - 1) {
        const int g = __ffs(left) - 1;
        const double other = __shfl_sync(kAll, mine, g);
        rank += other > mine || (other == mine && g < lane) ? 1 : 0;
    }
    return sure | __ballot_sync(kAll, ((near >> lane) & 1) && rank < p.topk_groups - __popc(sure));
}

// The choice by exact_keys(), pick by pick the best key after the last pick in the order (keys
// down, experts up).  Returns the experts of slots lane (low half) and lane + 32, 0xFFFF
// for none.  Below topk 32 about one token in a million comes here; from 32 on each one with a
// near tie among its picks, and at 64, where no slot is left for the first expert left out, each one
// unless bf16 logits decide alone (4096 tokens over 256 experts: topk 40 80 us, 64 353).
template <typename T>
__device__ __noinline__ uint32_t choose_exactly(const RouteParams &p, const T *row, double *s_key, int lane)
{
    const bool by_logit = p.bias == nullptr;
    const unsigned mask = exact_keys(p, row, s_key, lane);
    const int size = p.experts / p.groups;
    // (by logits the order is theirs, also where the groups went by scores)
    const bool from_row = by_logit && p.groups > 1 && p.group_top == 2;
    uint32_t pick0 = 0xFFFFu, pick1 = 0xFFFFu;
    uint64_t last = ~0ull;
    int last_i = -1;
#pragma unroll 1
    for (int r = 0; r < p.topk; ++r) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll 1
        for (int i = lane; i < p.experts; i += 32) {
            if (!((mask >> (i / size & 31)) & 1)) continue;
            const uint64_t k = ordered(from_row ? (double)clean(value_of(row[i])) : s_key[i]);
            if ((k < last || (k == last && i > last_i)) && k > best) { best = k; at = i; }
        }
        const uint64_t m = warp_max(best);
        if (m == 0) break;
        const int i = (int)__reduce_min_sync(kAll, best == m ? (unsigned)at : kAll);
        if (lane == r) pick0 = (uint32_t)i;
        if (lane == r - 32) pick1 = (uint32_t)i;
        last = m;
        last_i = i;
    }
    return pick0 | pick1 << 16;
}

// ------------------------------------------------------------- fast choice ----

// The experts [lane * V, lane * V + V) of a row, in vectors where `vec` (rows and V elements on
// boundaries of up to 16 bytes, experts a multiple of V).
template <int V, typename T>
__device__ __forceinline__ void load_row(const T *row, int lane, int experts, bool vec, float (&l)[V])
{
    constexpr int kBytes = V * (int)sizeof(T);
    const int first = lane * V;
    if (vec) {
        constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
        if (first < experts) {
            if constexpr (kBytes >= 16) {
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(row + first + i * (16 / (int)sizeof(T)));
                    w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
                }
            } else if constexpr (kBytes == 8) {
                const uint2 q = *reinterpret_cast<const uint2 *>(row + first);
                w[0] = q.x; w[1] = q.y;
            } else if constexpr (kBytes == 4) {
                w[0] = *reinterpret_cast<const uint32_t *>(row + first);
            } else {
                w[0] = *reinterpret_cast<const uint16_t *>(row + first);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f;
            if constexpr (sizeof(T) == 4) f = __uint_as_float(w[v]);
            else f = __uint_as_float(v & 1 ? w[v / 2] & 0xFFFF0000u : w[v / 2] << 16);
            l[v] = first < experts ? clean(f) : kNegInf;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = first + v < experts ? clean(value_of(row[first + v])) : kNegInf;
    }
}

// Descending order of V keys (Batcher's odd-even merge sort).
template <int V>
__device__ __forceinline__ void sort_descending(uint32_t (&k)[V])
{
#pragma unroll
    for (int p = 1; p < V; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t a = k[i + j], b = k[i + j + q];
                        k[i + j] = max(a, b);
                        k[i + j + q] = min(a, b);
                    }
}

__device__ __forceinline__ float key_of(const RouteParams &p, const Scores &score, float l, float b)
{
    return l > kNegInf && b > kNegInf ? score(l) + b : kNegInf;
}

// The two best of a group's keys, over the lanes of an aligned group of `lanes` lanes.
struct Top2 {
    float a, b;
    __device__ __forceinline__ void add(float k)
    {
        b = fmaxf(b, fminf(a, k));
        a = fmaxf(a, k);
    }
};

// A key and its expert as one word: the key's upper bits in the order of the floats, then the
// complement of the expert, so that a maximum finds the highest key, ties going to the
// lower expert.  Words of -inf are below kLowest, as is 0.
constexpr uint32_t kLowest = 0x00800000u;

template <int V>
__device__ __forceinline__ uint32_t word_of(float key, int expert)
{
    constexpr uint32_t kMask = 32 * V - 1;
    const int32_t u = __float_as_int(key + 0.0f);        // (-0 counts as 0)
    return ((uint32_t)(u ^ ((u >> 31) | (int32_t)0x80000000)) & ~kMask) | (kMask - (uint32_t)expert);
}

// The choice with fp32 keys, lane i owning the V experts from i V on.  A key and its expert
// are one word: the key's upper bits in the order of the floats, then the complement of
// the expert, so that one maximum over the warp finds a pick, ties going to the lower
// expert.  s_key: `experts` floats of the warp, for groups.  Each lane's words are sorted
// once, and a pick takes its lane's first one off.
// What the lower bits of the keys would have decided shows between neighbours in the
// order: false if two of them (or two groups) are too near each other for fp32, or
// sorted by the upper bits alone against their keys.
template <int V, typename T, bool kTwo>
__device__ __forceinline__ bool choose_fast(const RouteParams &p, const T *row, const float (&l)[V],
                                            const Scores &score, double *s_key, int lane, int (&pick)[2],
                                            float (&at)[2])
{
    float *const s_float = reinterpret_cast<float *>(s_key);
    constexpr uint32_t kMask = 32 * V - 1;
    const bool by_logit = p.bias == nullptr;
    const float rel = relative_error<V>(score.softmax);
    float key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = l[v];
    if (!by_logit) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane * V + v < p.experts) key[v] = key_of(p, score, l[v], p.bias[lane * V + v]);
    }
    if (p.groups > 1) {
        const int size = p.experts / p.groups, lanes = size / V;
        bool near = false;
        unsigned mask = 0;
        // groups of whole lanes, a power of two of them: by shuffles; others through shared memory, a
        // group per lane.  `mine`: the lane's group, `at0`: where group g's value stands, g * at0.
        const bool whole = lanes * V == size && (lanes & (lanes - 1)) == 0;
        Top2 top = {kNegInf, kNegInf};
        if (whole) {
#pragma unroll
            for (int v = 0; v < V; ++v) top.add(key[v]);
            for (int o = 1; o < lanes; o <<= 1) {
                const float a = __shfl_xor_sync(kAll, top.a, o), b = __shfl_xor_sync(kAll, top.b, o);
                top.b = fmaxf(fminf(top.a, a), fmaxf(top.b, b));
                top.a = fmaxf(top.a, a);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (lane * V + v < p.experts) s_float[lane * V + v] = key[v];
            __syncwarp();
            if (lane < p.groups)
                for (int i = 0; i < size; ++i) top.add(s_float[lane * size + i]);
            __syncwarp();
        }
        const int mine = whole ? lane / lanes : lane, at0 = whole ? lanes : 1;
        float value = top.a;
        if (p.group_top == 2 && top.a > kNegInf) {
            if (by_logit) value = score(top.a) + (top.b > kNegInf ? score(top.b) : 0.0f);
            else if (top.b > kNegInf) value = top.a + top.b;
        }
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float other = __shfl_sync(kAll, value, g * at0);
            rank += other > value || (other == value && g < mine) ? 1 : 0;
        }
        const bool here = mine < p.groups, kept = here && rank < p.topk_groups;
        if (!by_logit || p.group_top == 2) {
            // What a value may be off: its two scores (together at most 2, the softmax's 1), and three
            // roundings that go by the keys it is made of, which may cancel; nothing is known of
            // values past the floats but their side.
            const float keys = by_logit ? 2.0f : fmaxf(fabsf(top.a), p.group_top == 2 && top.b > kNegInf ? fabsf(top.b) : 0.0f);
            const float off = 2.0f * rel + 2.0f * kAbs + 8.0f * kRound * keys;
            float least = value - off, most = value + off;
            if (!(top.a > kNegInf)) least = most = kNegInf;
            else if (value == INFINITY) { least = 0x1.fp127f; most = INFINITY; }
            else if (value == kNegInf) { least = kNegInf; most = -0x1.fp127f; }
            // the lowest group that stays and the highest that does not
            const float low = -warp_max(kept ? -least : kNegInf), high = warp_max(here && !kept ? most : kNegInf);
            if (high > kNegInf && !(low > high)) {
                near = true;
                const int unsure = kept ? !(least > high) : here && !(low > most);
                const int state = __shfl_sync(kAll, (kept ? 1 : 0) | unsure << 1, lane * at0 & 31);
                const bool in = lane < p.groups;
                mask = exact_groups(p, row, __ballot_sync(kAll, in && (state & 1)), __ballot_sync(kAll, in && (state & 2)), lane);
            }
        }
        if (whole && !near) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (!kept) key[v] = kNegInf;
        } else {
            if (!near) mask = __ballot_sync(kAll, kept);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (!((mask >> ((lane * V + v) / size & 31)) & 1)) key[v] = kNegInf;
        }
    }
    uint32_t k[V];
#pragma unroll
    for (int v = 0; v < V; ++v) k[v] = word_of<V>(key[v], lane * V + v);
    sort_descending<V>(k);
    // a bf16 logit's bits are all among the upper ones
    const bool exact = by_logit && sizeof(T) == 2;
    uint32_t mine[2] = {0, 0};
    const int rounds = exact ? p.topk : p.topk + 1;
    for (int r = 0; r < rounds; ++r) {
        const uint32_t m = __reduce_max_sync(kAll, k[0]);
        mine[0] = lane == r ? m : mine[0];
        if constexpr (kTwo) mine[1] = lane == r - 32 ? m : mine[1];
        if (k[0] == m) {
#pragma unroll
            for (int v = 0; v + 1 < V; ++v) k[v] = k[v + 1];
            k[V - 1] = 0;
        }
    }
    float b[2] = {0.0f, 0.0f}, kf[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = mine[j] >= kLowest ? (int)(kMask - (mine[j] & kMask)) : -1;
        at[j] = i >= 0 ? clean(value_of(row[i])) : kNegInf;
        if (!by_logit && i >= 0) b[j] = p.bias[i];
        kf[j] = by_logit ? at[j] : key_of(p, score, at[j], b[j]);
        pick[j] = lane + 32 * j < p.topk ? i : -1;
        if constexpr (!kTwo) {                           // (one slot a lane, the first one left out among them)
            pick[1] = -1;
            at[1] = kNegInf;
            break;
        }
    }
    if (exact) return true;
    if (kTwo && p.topk >= 64) return false;
    // Slots past the picks: the first expert left out, and the next one's word.
    const uint32_t out_second = __reduce_max_sync(kAll, k[0]);
    if (out_second >= kLowest) {
        // It and all behind it are below every pick: below the lowest pick's key, which within one
        // prefix need not be the last slot's.  (Their scores are at most the row's highest.)
        const float next_most = unordered(out_second | kMask);
        float lowest = lane < p.topk ? kf[0] : INFINITY;
        if (kTwo && lane + 32 < p.topk) lowest = fminf(lowest, kf[1]);
        lowest = -warp_max(-lowest);
        const float most = score.softmax ? __fdividef(1.0f, score.sum) : 1.0f;
        const float tol = by_logit ? 0.0f : 2.0f * rel * most + 2.0f * kAbs + 2.0f * kRound * (fabsf(lowest) + fabsf(next_most));
        if (!(lowest - next_most > tol)) return false;
    }
    bool apart = true;                                   // neighbours are in order
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (j == 1 && !kTwo) break;
        uint32_t next = __shfl_down_sync(kAll, mine[j], 1);
        float next_at = __shfl_down_sync(kAll, at[j], 1), next_b = __shfl_down_sync(kAll, b[j], 1);
        float next_kf = __shfl_down_sync(kAll, kf[j], 1);
        if (j == 0 && kTwo) {
            const uint32_t n1 = __shfl_sync(kAll, mine[1], 0);
            const float a1 = __shfl_sync(kAll, at[1], 0), b1 = __shfl_sync(kAll, b[1], 0), k1 = __shfl_sync(kAll, kf[1], 0);
            if (lane == 31) { next = n1; next_at = a1; next_b = b1; next_kf = k1; }
        }
        const int slot = lane + 32 * j;
        if (slot >= p.topk || next < kLowest) continue;
        const float s = fmaxf(kf[j] - b[j], 0.0f) + fmaxf(next_kf - next_b, 0.0f);
        const float tol = by_logit ? 0.0f : rel * s + 2.0f * kAbs + 2.0f * kRound * (fabsf(kf[j]) + fabsf(next_kf));
        // (experts of one logit and one bias are equal in any precision)
        if (by_logit) apart = apart && at[j] >= next_at;
        else if (at[j] != next_at || b[j] != next_b || slot + 1 == p.topk) apart = apart && kf[j] - next_kf > tol;
    }
    if (__all_sync(kAll, apart)) return true;
    if (kTwo) return false;
    // The picks and the first one left out again by logits, or by keys in 64 bits: each one's
    // rank among them.  (With softmax scores and a bias all logits have to be read again for
    // their sum: 32768 tokens over 256 experts in 8 groups 49 us, 4096 ungrouped 13; a first form
    // by choose_exactly() took a third more and twice that.)
    const bool here = mine[0] >= kLowest && lane <= p.topk;
    const int expert = here ? (int)(kMask - (mine[0] & kMask)) : 32 * V;
    double exact_key = here ? (double)at[0] : (double)kNegInf;
    if (!by_logit) {
        const bool softmax = p.score == kScoreSoftmax;
        ExactSoftmax of = {0.0, 1.0};
        if (softmax) of = exact_softmax(p, row, lane);   // (two neighbours have a key)
        const double x = exp(softmax ? exact_key - of.max : -exact_key);
        if (here) exact_key = (softmax ? x / of.sum : 1.0 / (1.0 + x)) + (double)b[0];
    }
    int rank = 0;
    for (int i = 0; i <= p.topk; ++i) {
        const double other = __shfl_sync(kAll, exact_key, i);
        const int e = __shfl_sync(kAll, expert, i);
        rank += other > exact_key || (other == exact_key && e < expert) ? 1 : 0;
    }
    const float l0 = at[0];
    pick[0] = -1;
    at[0] = kNegInf;
    for (int i = 0; i <= p.topk; ++i) {
        const int r = __shfl_sync(kAll, rank, i), e = __shfl_sync(kAll, expert, i);
        const float l = __shfl_sync(kAll, l0, i);
        if (r == lane && lane < p.topk && e < 32 * V) {
            pick[0] = e;
            at[0] = l;
        }
    }
    return true;
}

// Lanes that hold the first topk slots, as a power of two (32 for more).
__device__ __forceinline__ int slot_lanes(int topk) { return topk <= 8 ? 8 : 32; }

__device__ __forceinline__ float slots_sum(float v, int lanes)
{
    for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Shares of the picks among themselves, their largest logit `top` taken out: a softmax over them,
// or s / e^min(top, 0) for the sigmoid, neither of which underflows in all.
__device__ __forceinline__ float share_of(bool softmax, float at, float top)
{
    if (softmax) return expf(at - top);
    if (top < 0.0f) return __fdividef(expf(at - top), 1.0f + expf(at));
    const float t = expf(-fabsf(at));
    return __fdividef(at > 0.0f ? 1.0f : t, 1.0f + t);
}

template <bool kTwo>
__device__ __forceinline__ void shares(bool softmax, const int (&pick)[2], const float (&at)[2], int topk, float (&u)[2])
{
    const float top = unordered(__reduce_max_sync(kAll, max(ordered(at[0]), kTwo ? ordered(at[1]) : 0u)));
    u[0] = pick[0] >= 0 ? share_of(softmax, at[0], top) : 0.0f;
    u[1] = kTwo && pick[1] >= 0 ? share_of(softmax, at[1], top) : 0.0f;
    const float sum = slots_sum(u[0] + u[1], slot_lanes(topk));
    u[0] = pick[0] >= 0 ? __fdividef(u[0], sum) : 0.0f;
    if constexpr (kTwo) u[1] = pick[1] >= 0 ? __fdividef(u[1], sum) : 0.0f;
}

// The choice by whole logits, where words of one prefix may be sorted against them: pick by
// pick the best after the last one in the order (logits down, experts up).  Small, as it is
// cold when it is called.
template <typename T>
__device__ __forceinline__ int choose_by_logit(const RouteParams &p, const T *row, int lane)
{
    int pick = -1, last_i = -1;
    uint32_t last = ~0u;
#pragma unroll 1
    for (int r = 0; r < p.topk; ++r) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll 1
        for (int i = lane; i < p.experts; i += 32) {
            const uint32_t k = ordered(clean(value_of(row[i])));
            if ((k < last || (k == last && i > last_i)) && k > best) { best = k; at = i; }
        }
        const uint32_t m = __reduce_max_sync(kAll, best);
        if (m == 0) break;
        const int i = (int)__reduce_min_sync(kAll, best == m ? (unsigned)at : kAll);
        pick = lane == r ? i : pick;
        last = m;
        last_i = i;
    }
    return pick;
}

// Routing without bias and groups, topk below 32 (a slot a lane, the first expert left out
// among them): the order of the logits decides, and nothing of the rest is in the
// registers or the code (16384 tokens, top 8 of 128: 500 instructions a token in the
// general kernel).
template <int V, typename T>
__global__ void __launch_bounds__(32 * kWarps) moe_route_plain_kernel(const RouteParams p, bool vec)
{
    constexpr uint32_t kMask = 32 * V - 1;
    constexpr bool kExact = sizeof(T) == 2;              // (a bf16 logit's bits are all in the word)
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= (uint32_t)p.tokens) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.ldl;
    uint32_t k[V];
    Scores score = {p.score == kScoreSoftmax, 0.0f, 1.0f};
    {
        float l[V];
        load_row<V, T>(row, lane, p.experts, vec, l);
        if (score.softmax && !p.renorm) score = scores_of<V>(p, l);
#pragma unroll
        for (int v = 0; v < V; ++v) k[v] = word_of<V>(l[v], lane * V + v);
    }
    sort_descending<V>(k);
    uint32_t mine = 0;
    const int rounds = kExact ? p.topk : p.topk + 1;
    for (int r = 0; r < rounds; ++r) {
        const uint32_t m = __reduce_max_sync(kAll, k[0]);
        mine = lane == r ? m : mine;
        if (k[0] == m) {
#pragma unroll
            for (int v = 0; v + 1 < V; ++v) k[v] = k[v + 1];
            k[V - 1] = 0;
        }
    }
    int pick = mine >= kLowest ? (int)(kMask - (mine & kMask)) : -1;
    float at = pick >= 0 ? clean(value_of(row[pick])) : kNegInf;
    if constexpr (!kExact) {
        // words of one prefix may be sorted against their logits: the picks and the first one
        // left out are ranked again; if the next one shares the last pick's prefix, all are
        const uint32_t last = __shfl_sync(kAll, mine, p.topk - 1), second = __reduce_max_sync(kAll, k[0]);
        const float next = __shfl_down_sync(kAll, at, 1);
        if (second >= kLowest && ((last ^ second) & ~kMask) == 0) {
            pick = choose_by_logit(p, row, lane);
            at = pick >= 0 ? clean(value_of(row[pick])) : kNegInf;
        } else if (__any_sync(kAll, lane < p.topk && pick >= 0 && !(at >= next))) {
            const uint32_t key = pick >= 0 ? ordered(at) : 0u;
            int rank = 0, to = -1;
            for (int i = 0; i <= p.topk; ++i) {
                const uint32_t other = __shfl_sync(kAll, key, i);
                const int e = __shfl_sync(kAll, pick, i);
                rank += other > key || (other == key && e < pick) ? 1 : 0;
            }
            for (int i = 0; i <= p.topk; ++i) {
                const int r = __shfl_sync(kAll, rank, i), e = __shfl_sync(kAll, pick, i);
                if (r == lane && e >= 0) to = e;
            }
            pick = to;
            at = pick >= 0 ? clean(value_of(row[pick])) : kNegInf;
        }
        if (lane >= p.topk) pick = -1;
    }
    float w;
    if (p.renorm) {
        const float top = __shfl_sync(kAll, at, 0);      // (the first pick's logit is the largest)
        const float u = pick >= 0 ? share_of(score.softmax, at, top) : 0.0f;
        w = __fdividef(u, slots_sum(u, slot_lanes(p.topk)));
    } else {
        w = score(at);
    }
    if (lane < p.topk) {
        const int64_t o = (int64_t)t * p.topk + lane;
        p.ids[o] = pick;
        p.weights[o] = pick >= 0 ? p.scale * w : 0.0f;
    }
}

// kTwo: two slots a lane, for topk of 32 and more.
template <int V, typename T, bool kTwo>
__global__ void __launch_bounds__(32 * kWarps) moe_route_kernel(const __grid_constant__ RouteParams p, bool vec)
{
    extern __shared__ double s_keys[];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= p.tokens) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.ldl;
    float l[V];
    load_row<V, T>(row, lane, p.experts, vec, l);
    const bool softmax = p.score == kScoreSoftmax;
    Scores score = {softmax, 0.0f, 1.0f};
    if (softmax && (!p.renorm || p.bias != nullptr || (p.groups > 1 && p.group_top == 2))) score = scores_of<V>(p, l);
    int pick[2];
    float at[2], w[2];
    double *const s_key = s_keys + warp * p.experts;
    if (!choose_fast<V, T, kTwo>(p, row, l, score, s_key, lane, pick, at)) {
        const uint32_t found = choose_exactly(p, row, s_key, lane);
        pick[0] = (found & 0xFFFFu) == 0xFFFFu ? -1 : (int)(found & 0xFFFFu);
        pick[1] = found >> 16 == 0xFFFFu ? -1 : (int)(found >> 16);
#pragma unroll
        for (int j = 0; j < 2; ++j) at[j] = pick[j] >= 0 ? clean(value_of(row[pick[j]])) : kNegInf;
    }
#pragma unroll
    for (int j = 0; j < (kTwo ? 2 : 1); ++j)
        if (pick[j] < 0) at[j] = kNegInf;
    if (p.renorm) {
        shares<kTwo>(softmax, pick, at, p.topk, w);
    } else {
        w[0] = score(at[0]);
        if constexpr (kTwo) w[1] = score(at[1]);
    }
#pragma unroll
    for (int j = 0; j < (kTwo ? 2 : 1); ++j)
        if (lane + 32 * j < p.topk) {
            p.ids[t * p.topk + lane + 32 * j] = pick[j];
            p.weights[t * p.topk + lane + 32 * j] = pick[j] >= 0 ? p.scale * w[j] : 0.0f;
        }
}

// ---------------------------------------------------------------- gradient ----
// s (1 - s) of a sigmoid.
__device__ __forceinline__ float slope_of(float l)
{
    const float t = expf(-fabsf(l)), r = reciprocal(1.0f + t);
    return t * r * r;
}

// With g_j = scale * dweights_j of pick j (expert i_j) and u the shares of the picks:
//   softmax, renormalised  d_j = u_j (g_j - sum_k u_k g_k)
//   sigmoid, renormalised  d_j = (1 - s_j) u_j (g_j - sum_k u_k g_k)
//   sigmoid                d_j = g_j s_j (1 - s_j)
//   softmax                picked:  s_i (G_i - sum_k s_k G_k), others: -s_i sum_k s_k G_k
// where G merges picks of one expert.  The gradients enter less that of the pick of the
// largest weight (which changes nothing: the weights sum to 1, for the plain softmax with
// the others' mass), so that nothing cancels where one pick has nearly all the weight.
template <int V, typename T, bool kTwo>
__global__ void __launch_bounds__(32 * kWarps) moe_route_backward_kernel(const RouteParams p, bool vec)
{
    __shared__ __align__(16) float s_rows[kWarps][32 * V];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= p.tokens) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.ldl;
    const bool softmax = p.score == kScoreSoftmax, dense = softmax && !p.renorm;
    const int lanes = slot_lanes(p.topk);
    int pick[2] = {-1, -1};
    float at[2] = {kNegInf, kNegInf}, g[2] = {0.0f, 0.0f}, u[2] = {0.0f, 0.0f}, d[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int slot = lane + 32 * j;
        if (slot >= p.topk || (j == 1 && !kTwo)) break;
        const int id = p.ids[t * p.topk + slot];
        const float dw = p.dw[t * p.topk + slot];
        if (id < 0 || id >= p.experts) continue;
        at[j] = clean(value_of(row[id]));
        if (!(at[j] > kNegInf)) continue;
        pick[j] = id;
        g[j] = p.scale * dw;
    }
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    // picks of one expert: of lanes that name it only one finds its mark (two slots a lane:
    // not looked for)
    float *const s_row = s_rows[warp];
    bool repeated = kTwo;
    if constexpr (!kTwo) {
        if (pick[0] >= 0) reinterpret_cast<volatile int *>(s_row)[pick[0]] = lane;
        __syncwarp();
        repeated = __any_sync(kAll, pick[0] >= 0 && reinterpret_cast<volatile int *>(s_row)[pick[0]] != lane);
    }
    if (p.renorm) {
        shares<kTwo>(softmax, pick, at, p.topk, u);
    } else if (dense) {
        float l[V];
        load_row<V, T>(row, lane, p.experts, vec, l);
        const Scores score = scores_of<V>(p, l);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = l[v] > kNegInf ? score(l[v]) : 0.0f;
        if (repeated) {                                  // the first carries their sum
            float merged[2] = {0.0f, 0.0f};
            bool first[2] = {true, true};
            for (int k = 0; k < p.topk; ++k) {
                const int id = __shfl_sync(kAll, pick[kTwo ? k >> 5 : 0], k & 31);
                const float gk = __shfl_sync(kAll, g[kTwo ? k >> 5 : 0], k & 31);
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
            }
        }
        u[0] = pick[0] >= 0 ? score(at[0]) : 0.0f;
        if constexpr (kTwo) u[1] = pick[1] >= 0 ? score(at[1]) : 0.0f;
    } else {
        if (pick[0] >= 0) d[0] = g[0] * slope_of(at[0]);
        if (kTwo && pick[1] >= 0) d[1] = g[1] * slope_of(at[1]);
    }
    float mean = 0.0f, ref = 0.0f;
    if (p.renorm || dense) {
        // (shares are not negative: their bits are in order)
        const uint32_t best = __reduce_max_sync(kAll, __float_as_uint(fmaxf(u[0], u[1])));
        const bool has0 = __float_as_uint(u[0]) == best;
        const unsigned who = __ballot_sync(kAll, has0 || __float_as_uint(u[1]) == best);
        ref = __shfl_sync(kAll, has0 ? g[0] : g[1], __ffs(who) - 1);
        mean = slots_sum((u[0] > 0.0f ? u[0] * (g[0] - ref) : 0.0f) + (u[1] > 0.0f ? u[1] * (g[1] - ref) : 0.0f), lanes);
        mean = __shfl_sync(kAll, mean, 0);
    }
    if (p.renorm) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (pick[j] >= 0) {
                d[j] = u[j] * ((g[j] - ref) - mean);
                if (!softmax) d[j] *= reciprocal(1.0f + expf(at[j]));
            }
    } else if (dense) {
        // sum_k s_k G_k = ref (1 - rest) + mean, rest the mass of the others: picked ones have
        // s_i ((G_i - ref) - mean + ref rest), others -s_i (ref (1 - rest) + mean)
        unsigned taken[(V + 31) / 32] = {};
        for (int k = 0; k < p.topk; ++k) {
            const int id = __shfl_sync(kAll, pick[kTwo ? k >> 5 : 0], k & 31) - lane * V;
            if (id >= 0 && id < V) taken[0] |= 1u << id;
        }
        float others = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (!((taken[0] >> v) & 1)) others += acc[v];
        others = warp_sum(others);
        const float dot = __shfl_sync(kAll, slots_sum(u[0] * g[0] + u[1] * g[1], lanes), 0);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = (taken[0] >> v) & 1 ? 0.0f : -acc[v] * dot;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (pick[j] >= 0) d[j] = u[j] * ((g[j] - ref) - mean + ref * others);
    }
    // the picks' gradients to their places among the lane's V
    if (!repeated || dense) {
#pragma unroll
        for (int v = 0; v < V; ++v) s_row[lane * V + v] = acc[v];
        __syncwarp();
        if (pick[0] >= 0) s_row[pick[0]] = d[0];
        if (kTwo && pick[1] >= 0) s_row[pick[1]] = d[1];
        __syncwarp();
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = s_row[lane * V + v];
    } else {                                             // in the order of the slots
        for (int k = 0; k < p.topk; ++k) {
            const int id = __shfl_sync(kAll, pick[kTwo ? k >> 5 : 0], k & 31) - lane * V;
            const float dk = __shfl_sync(kAll, d[kTwo ? k >> 5 : 0], k & 31);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (id == v) acc[v] += dk;
        }
    }
    T *out = static_cast<T *>(p.dlogits) + t * p.ldd + lane * V;
    if (vec) {
        if (lane * V < p.experts) store_vector<V, T>(out, acc);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane * V + v < p.experts) store_value(out + v, acc[v]);
    }
}

cudaError_t launch_dependent(void (*kernel)(RouteParams, bool), size_t smem, bool vec, cudaStream_t s, const RouteParams &p)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(((int64_t)p.tokens + kWarps - 1) / kWarps), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, vec);
}

using Kernel = void (*)(RouteParams, bool);

enum Kind { kGeneral, kPlain, kBackward };

template <typename T, int V>
constexpr Kernel kernel_of(Kind kind, bool two)
{
    // (32 experts and fewer have no second slots, but for topk = 32 of them)
    return kind == kBackward ? (two ? moe_route_backward_kernel<V, T, true> : moe_route_backward_kernel<V, T, false>)
           : kind == kPlain  ? moe_route_plain_kernel<V, T>
           : two             ? moe_route_kernel<V, T, true>
                             : moe_route_kernel<V, T, false>;
}

// Experts per lane: the power of two that holds them all.
int lane_experts(int experts)
{
    int v = 1;
    while (32 * v < experts) v *= 2;
    return v;
}

template <typename T>
Kernel kernel_for(int v, Kind kind, bool two)
{
    return v == 1    ? kernel_of<T, 1>(kind, two)
           : v == 2  ? kernel_of<T, 2>(kind, two)
           : v == 4  ? kernel_of<T, 4>(kind, two)
           : v == 8  ? kernel_of<T, 8>(kind, two)
           : v == 16 ? kernel_of<T, 16>(kind, two)
                     : kernel_of<T, 32>(kind, two);
}

bool vector_rows(const void *base, int64_t ld, int size, int v, int experts)
{
    const int bytes = std::min(16, v * size);
    return experts % v == 0 && reinterpret_cast<uintptr_t>(base) % bytes == 0 && ld * size % bytes == 0;
}

}  // namespace

cudaError_t launch_route(const RouteParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    const int v = lane_experts(p.experts), size = p.type == kTypeF32 ? 4 : 2;
    const Kind kind = p.bias == nullptr && p.groups == 1 && p.topk < 32 ? kPlain : kGeneral;
    const size_t smem = kind == kGeneral ? (size_t)kWarps * p.experts * sizeof(double) : 0;
    return launch_dependent(size == 4 ? kernel_for<float>(v, kind, p.topk >= 32) : kernel_for<uint16_t>(v, kind, p.topk >= 32), smem,
                            vector_rows(p.logits, p.ldl, size, v, p.experts), s, p);
}

cudaError_t launch_route_backward(const RouteParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    const int v = lane_experts(p.experts), size = p.type == kTypeF32 ? 4 : 2;
    const bool vec = vector_rows(p.logits, p.ldl, size, v, p.experts) && vector_rows(p.dlogits, p.ldd, size, v, p.experts);
    return launch_dependent(size == 4 ? kernel_for<float>(v, kBackward, p.topk > 32)
                                      : kernel_for<uint16_t>(v, kBackward, p.topk > 32), 0, vec, s, p);
}

}  // namespace nvfp4
