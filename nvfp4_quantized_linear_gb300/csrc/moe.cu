// Token movement of a mixture-of-experts layer around the grouped GEMM.
//
//   sort      row of assignment (t, k) in groups by expert, each group padded
//             to 128 rows (the grouped GEMM's layout), tokens in order
//   dispatch  rows[dest[t, k]] = x[t], as bf16 or quantized to NVFP4
//   combine   out[t] = sum_k w[t, k] * y[dest[t, k]] (+ residual[t])
//   backward of combine: dy[dest[t, k]] = w[t, k] * g[t],
//                        dw[t, k] = sum_h g[t, h] * y[dest[t, k], h]
// The gradient of dispatch is combine without weights.  Every kernel but the
// sort is a stream over rows: bytes bound it.  No atomics on values anywhere:
// sums run over k in order, so results do not depend on scheduling.
#include <cuda_bf16.h>

#include "block_launch.cuh"
#include "common.cuh"
#include "ptx.cuh"
#include "quant_core.cuh"
#include "scale_math.cuh"

namespace nvfp4 {
namespace {

using namespace quant_core;

// ------------------------------------------------------------------- sort ----
// A stable counting sort.  Block b owns a range of whole 1024-assignment tiles.
// moe_count_kernel: the block's count per expert.  moe_place_kernel: the sum of
// the preceding blocks' counts, the group offsets (every block computes them
// alike from all counts) and, tile by tile, each assignment's rank among the
// block's earlier ones of its expert: inside a warp by matching lanes, across
// warps by a prefix over the warps' counts.

template <typename Id>
__device__ __forceinline__ int load_id(const void *ids, int64_t i, int n, int experts)
{
    if (i >= n) return -1;
    const Id v = static_cast<const Id *>(ids)[i];
    return v >= 0 && v < (Id)experts ? (int)v : -1;
}

template <typename Id>
__global__ void __launch_bounds__(kMoeSortTile) moe_count_kernel(const MoeSortParams p, int tiles_per_block)
{
    __shared__ int s_count[kMoeMaxExperts];
    for (int e = threadIdx.x; e < p.experts; e += kMoeSortTile) s_count[e] = 0;
    __syncthreads();
    for (int t = 0; t < tiles_per_block; ++t) {
        const int64_t i = ((int64_t)blockIdx.x * tiles_per_block + t) * kMoeSortTile + threadIdx.x;
        const int id = load_id<Id>(p.ids, i, p.n, p.experts);
        if (id >= 0) atomicAdd(&s_count[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kMoeSortTile) p.hist[(int64_t)blockIdx.x * p.experts + e] = s_count[e];
}

template <typename Id>
__global__ void __launch_bounds__(kMoeSortTile) moe_place_kernel(const MoeSortParams p, int tiles_per_block)
{
    extern __shared__ uint16_t s_warp[];                 // [32 warps][experts] counts of a tile
    __shared__ int s_next[kMoeMaxExperts];               // next row of each expert for this block
    __shared__ int s_scan[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int experts = p.experts;
    int before = 0, total = 0;                           // expert tid: rows of earlier blocks, of all
    if (tid < experts)
        for (int b = 0; b < (int)gridDim.x; ++b) {
            const int c = p.hist[(int64_t)b * experts + tid];
            if (b < (int)blockIdx.x) before += c;
            total += c;
        }
    const int padded = (total + 127) / 128 * 128;
    int incl = padded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += s_scan[w];
    const int offset = base + incl - padded;
    if (tid < experts) {
        s_next[tid] = offset + before;
        if (blockIdx.x == 0) {
            p.offsets[tid] = offset;
            p.counts[tid] = total;
            if (tid == experts - 1) p.offsets[experts] = offset + padded;
        }
    }
    for (int t = 0; t < tiles_per_block; ++t) {
        const int64_t i = ((int64_t)blockIdx.x * tiles_per_block + t) * kMoeSortTile + tid;
        for (int j = tid; j < 32 * experts; j += kMoeSortTile) s_warp[j] = 0;
        __syncthreads();
        const int id = load_id<Id>(p.ids, i, p.n, experts);
        const unsigned peers = __match_any_sync(kFull, id);
        const int rank = __popc(peers & ((1u << lane) - 1));
        if (id >= 0 && rank == 0) s_warp[warp * experts + id] = (uint16_t)__popc(peers);
        __syncthreads();
        if (tid < experts) {                             // exclusive prefix over the warps; advance the expert
            int run = 0;
            for (int w = 0; w < 32; ++w) {
                const int c = s_warp[w * experts + tid];
                s_warp[w * experts + tid] = (uint16_t)run;
                run += c;
            }
            total = run;
        }
        __syncthreads();
        if (i < p.n) p.dest[i] = id < 0 ? -1 : s_next[id] + s_warp[warp * experts + id] + rank;
        __syncthreads();
        if (tid < experts) s_next[tid] += total;
    }
}

// --------------------------------------------------------------- dispatch ----
// Blocks [0, tokens): a token's row to its assignments' rows, read once.
// Blocks past them, one per expert: zeros into the group's padding rows.

__device__ __forceinline__ uint4 load8(const uint16_t *row, int c, int h)
{
    if (c + 8 <= h) return *reinterpret_cast<const uint4 *>(row + c);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = c + i < h ? row[c + i] : 0u;
    return make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
}

__device__ __forceinline__ void store8(uint16_t *row, int c, int h, const uint4 &v)
{
    if (c + 8 <= h) {
        *reinterpret_cast<uint4 *>(row + c) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < h) row[c + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

// Row of an assignment, -1 for a dropped one (or one that the buffer of
// p.rows rows does not hold).
__device__ __forceinline__ int row_of(const MoeRowsParams &p, int64_t assignment)
{
    const int d = __ldg(p.dest + assignment);
    return d < p.rows ? d : -1;
}

__device__ __forceinline__ void zero_padding_rows(const MoeRowsParams &p, int e)
{
    const int first = max(0, p.offsets[e] + p.counts[e]), end = min(p.offsets[e + 1], p.rows);
    for (int r = first; r < end; ++r)
        for (int c = threadIdx.x * 8; c < p.h; c += blockDim.x * 8)
            store8(p.out + (int64_t)r * p.ldo, c, p.h, make_uint4(0, 0, 0, 0));
}

__global__ void __launch_bounds__(256) moe_dispatch_kernel(const MoeRowsParams p)
{
    if ((int)blockIdx.x >= p.tokens) {
        zero_padding_rows(p, blockIdx.x - p.tokens);
        return;
    }
    const int64_t first = (int64_t)blockIdx.x * p.topk;     // the token's assignments
    const uint16_t *x = p.x + (int64_t)blockIdx.x * p.ldx;
    for (int c = threadIdx.x * 8; c < p.h; c += blockDim.x * 8) {
        const uint4 v = load8(x, c, p.h);
        for (int k = 0; k < p.topk; ++k) {
            const int d = row_of(p, first + k);
            if (d >= 0) store8(p.out + (int64_t)d * p.ldo, c, p.h, v);
        }
    }
}

// The same with the row quantized to NVFP4 on the way: one thread per
// 16-element block, four neighbours' scale codes stored as one word.
__global__ void __launch_bounds__(256) moe_dispatch_quant_kernel(const MoeRowsParams p)
{
    const int64_t first = (int64_t)blockIdx.x * p.topk;     // the token's assignments
    const uint16_t *x = p.x + (int64_t)blockIdx.x * p.ldx;
    const float gs = __ldg(p.gs);
    const int steps = (p.nbp + blockDim.x - 1) / blockDim.x;
    for (int u = 0; u < steps; ++u) {
        const int blk = u * blockDim.x + threadIdx.x;
        const int k0 = blk * 16;
        const Raw16 raw = load16(x, k0, p.h, k0 < p.h);
        float v0[8], v1[8];
        unpack8(raw.a, v0);
        unpack8(raw.b, v1);
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max_abs3(amax, v0[i], v1[i]);
        const uint32_t code = cvt_e4m3x2(0.0f, div6_rn(__fmul_rn(amax, gs))) & 0x7Fu;
        const float d = e4m3_to_f32(code);
        const float inv = d == 0.0f ? 0.0f : __fdiv_rn(gs, d);
        const uint2 q = make_uint2(quant8(v0, inv), quant8(v1, inv));
        const uint32_t c1 = __shfl_down_sync(kFull, code, 1);
        const uint32_t c2 = __shfl_down_sync(kFull, code, 2);
        const uint32_t c3 = __shfl_down_sync(kFull, code, 3);
        const uint32_t word = code | (c1 << 8) | (c2 << 16) | (c3 << 24);
        for (int k = 0; k < p.topk; ++k) {
            const int r = row_of(p, first + k);
            if (r < 0) continue;
            if (blk < p.nb) *reinterpret_cast<uint2 *>(p.q + (int64_t)r * (p.kp / 2) + k0 / 2) = q;
            if ((threadIdx.x & 3) == 0 && blk < p.nb)
                *reinterpret_cast<uint32_t *>(p.sf + sf_offset(r, blk, p.nbp)) = word;
        }
    }
}

// ---------------------------------------------------------------- combine ----
__global__ void __launch_bounds__(256) moe_combine_kernel(const MoeRowsParams p)
{
    const int64_t t = blockIdx.x;
    for (int c = threadIdx.x * 8; c < p.h; c += blockDim.x * 8) {
        float acc[8] = {};
        for (int k = 0; k < p.topk; ++k) {
            const int r = row_of(p, t * p.topk + k);
            if (r < 0) continue;
            float v[8];
            unpack8(load8(p.x + (int64_t)r * p.ldx, c, p.h), v);
            const float w = p.weights != nullptr ? p.weights[t * p.topk + k] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(w, v[i], acc[i]);
        }
        if (p.residual != nullptr) {
            float v[8];
            unpack8(load8(p.residual + t * p.ldr, c, p.h), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += v[i];
        }
        store8(p.out + t * p.ldo, c, p.h, make_uint4(bf16x2_rn(acc[0], acc[1]), bf16x2_rn(acc[2], acc[3]),
                                                     bf16x2_rn(acc[4], acc[5]), bf16x2_rn(acc[6], acc[7])));
    }
}

// Blocks as in moe_dispatch_kernel.  Each assignment in turn: its dot product
// (fp32; lanes, then warps, in a fixed order) and its gradient row.
__global__ void __launch_bounds__(256) moe_combine_backward_kernel(const MoeRowsParams p)
{
    if ((int)blockIdx.x >= p.tokens) {
        zero_padding_rows(p, blockIdx.x - p.tokens);
        return;
    }
    __shared__ float s_dot[8];
    const int64_t t = blockIdx.x;
    const uint16_t *g = p.g + t * p.ldg;
    for (int k = 0; k < p.topk; ++k) {
        const int r = row_of(p, t * p.topk + k);
        float dot = 0.0f;
        if (r >= 0) {
            const float w = p.weights[t * p.topk + k];
            for (int c = threadIdx.x * 8; c < p.h; c += blockDim.x * 8) {
                float a[8], y[8];
                unpack8(load8(g, c, p.h), a);
                unpack8(load8(p.x + (int64_t)r * p.ldx, c, p.h), y);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot = __fmaf_rn(a[i], y[i], dot);
                    a[i] *= w;
                }
                store8(p.out + (int64_t)r * p.ldo, c, p.h, make_uint4(bf16x2_rn(a[0], a[1]), bf16x2_rn(a[2], a[3]),
                                                                      bf16x2_rn(a[4], a[5]), bf16x2_rn(a[6], a[7])));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
        if ((threadIdx.x & 31) == 0) s_dot[threadIdx.x >> 5] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = 0.0f;
            for (int w = 0; w < 8; ++w) sum += s_dot[w];
            p.dw[t * p.topk + k] = sum;
        }
        __syncthreads();
    }
}

template <typename Id>
cudaError_t launch_sort(const MoeSortParams &p, int num_sms, cudaStream_t s)
{
    const int tiles = p.n > 0 ? (p.n + kMoeSortTile - 1) / kMoeSortTile : 1;   // (no tokens: the offsets are still written)
    const int per_block = (tiles + num_sms - 1) / num_sms;
    const int blocks = (tiles + per_block - 1) / per_block;
    const size_t smem = (size_t)32 * p.experts * sizeof(uint16_t);
    if (smem > 48 * 1024 - sizeof(int) * (kMoeMaxExperts + 32)) {
        cudaError_t e = cudaFuncSetAttribute(moe_place_kernel<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    moe_count_kernel<Id><<<blocks, kMoeSortTile, 0, s>>>(p, per_block);
    moe_place_kernel<Id><<<blocks, kMoeSortTile, smem, s>>>(p, per_block);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_sort(const MoeSortParams &p, int num_sms, cudaStream_t s)
{
    return p.id_bytes == 8 ? launch_sort<int64_t>(p, num_sms, s) : launch_sort<int32_t>(p, num_sms, s);
}

cudaError_t launch_moe_dispatch(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    moe_dispatch_kernel<<<(unsigned)(p.tokens + p.experts), 256, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_moe_dispatch_quant(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    moe_dispatch_quant_kernel<<<(unsigned)p.tokens, 256, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_moe_combine(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    moe_combine_kernel<<<(unsigned)p.tokens, 256, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_moe_combine_backward(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    moe_combine_backward_kernel<<<(unsigned)(p.tokens + p.experts), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace nvfp4
