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
#include <algorithm>

#include <cuda_bf16.h>

#include "block_launch.cuh"
#include "common.cuh"
#include "epilogue.cuh"
#include "ptx.cuh"
#include "quant_core.cuh"
#include "scale_math.cuh"

namespace nvfp4 {
namespace {

using namespace quant_core;

// Up to here one cluster sorts in one launch, a block per tile (2048 assignments
// over 64 experts: 3.2 us, 5.0 by one block; 8192 over 32: 3.2, in two launches
// 4.4; 16384 over 64 with two tiles per block, which count before they rank: 6.2
// and 4.9).
constexpr int kClusterTiles = 8;

// ------------------------------------------------------------------- sort ----
// A stable counting sort.  Block b owns a range of whole 1024-assignment tiles.
// moe_count_kernel (more than kClusterTiles tiles): the block's count per expert.
// moe_place_kernel: the sum of
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

// Word of a cluster block's shared memory (address from mapa_shared).
__device__ __forceinline__ int ld_dsmem_s32(uint32_t addr)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <typename Id>
__global__ void __launch_bounds__(kMoeSortTile) moe_count_kernel(const MoeSortParams p, int tiles_per_block)
{
    __shared__ int s_count[kMoeMaxExperts];
    griddep_launch_dependents();
    for (int e = threadIdx.x; e < p.experts; e += kMoeSortTile) s_count[e] = 0;
    griddep_wait();
    __syncthreads();
    for (int t = 0; t < tiles_per_block; ++t) {
        const int64_t i = ((int64_t)blockIdx.x * tiles_per_block + t) * kMoeSortTile + threadIdx.x;
        const int id = load_id<Id>(p.ids, i, p.n, p.experts);
        if (id >= 0) atomicAdd(&s_count[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kMoeSortTile) p.hist[(int64_t)blockIdx.x * p.experts + e] = s_count[e];
}

// kCluster: the blocks of one cluster, a tile each, sort everything in one launch; a
// block reads the others' counts from their shared memory.
template <typename Id, bool kCluster>
__global__ void __launch_bounds__(kMoeSortTile) moe_place_kernel(const MoeSortParams p, int tiles_per_block)
{
    extern __shared__ uint16_t s_warp[];                 // [32 warps][experts] counts of a tile
    __shared__ int s_next[kMoeMaxExperts];               // next row of each expert for this block
    __shared__ int s_total[kMoeMaxExperts];              // (of the block's tile in a cluster)
    __shared__ int s_scan[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int experts = p.experts;
    auto clear_warps = [&] {
        for (int j = tid; j < 16 * experts; j += kMoeSortTile) reinterpret_cast<uint32_t *>(s_warp)[j] = 0;
    };
    // ranks the tile's ids: the thread's rank among its warp's equal ones, in
    // s_warp the count in the warps before (cleared at the call), and as result
    // the tile's count of expert tid
    int rank = 0;
    auto rank_tile = [&](int id) {
        const unsigned peers = __match_any_sync(kFull, id);
        rank = __popc(peers & ((1u << lane) - 1));
        if (id >= 0 && rank == 0) s_warp[warp * experts + id] = (uint16_t)__popc(peers);
        __syncthreads();
        int run = 0;
        if (tid < experts) {                             // exclusive prefix over the warps
#pragma unroll 8
            for (int w = 0; w < 32; ++w) {
                const int c = s_warp[w * experts + tid];
                s_warp[w * experts + tid] = (uint16_t)run;
                run += c;
            }
        }
        return run;
    };
    griddep_launch_dependents();
    for (int e = tid; e < experts; e += kMoeSortTile) s_next[e] = s_total[e] = 0;
    clear_warps();
    const int64_t first = (int64_t)blockIdx.x * tiles_per_block * kMoeSortTile;
    griddep_wait();
    int id = load_id<Id>(p.ids, first + tid, p.n, experts);       // the first tile's, with the counts in flight
    __syncthreads();
    int total = 0, run = 0;
    if constexpr (kCluster) {
        run = rank_tile(id);
        if (tid < experts) s_total[tid] = run;
        cluster_arrive_release();
        cluster_wait_acquire();
        if (tid < experts) {
            int before = 0;
#pragma unroll
            for (int r = 0; r < kClusterTiles; ++r) {
                const int c = r < (int)gridDim.x ? ld_dsmem_s32(mapa_shared(&s_total[tid], r)) : 0;
                before += r < (int)blockIdx.x ? c : 0;
                total += c;
            }
            s_next[tid] = before;
        }
        cluster_arrive_release();                        // (waited for at the end: the counts outlive their readers)
    } else {
        // column sums of hist: `groups` threads per expert, each a share of the
        // blocks (integer adds: their order does not matter)
        const int width = (experts + 31) / 32 * 32, groups = kMoeSortTile / width;
        const int e = tid % width, g = tid / width;
        if (e < experts && g < groups) {
            int before = 0, sum = 0;
#pragma unroll 16
            for (int b = g; b < (int)gridDim.x; b += groups) {
                const int c = p.hist[(int64_t)b * experts + e];
                before += b < (int)blockIdx.x ? c : 0;
                sum += c;
            }
            if (sum) atomicAdd(&s_total[e], sum);
            if (before) atomicAdd(&s_next[e], before);
        }
        __syncthreads();
        if (tid < experts) total = s_total[tid];
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
    int base = lane < warp ? s_scan[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(kFull, base, o);
    const int offset = base + incl - padded;
    if (tid < experts) {
        s_next[tid] += offset;
        if (blockIdx.x == 0) {
            p.offsets[tid] = offset;
            p.counts[tid] = total;
            if (tid == experts - 1) p.offsets[experts] = offset + padded;
        }
    }
    for (int t = 0; t < tiles_per_block; ++t) {
        const int64_t i = first + t * kMoeSortTile + tid;
        if (!kCluster) {
            if (t > 0) id = load_id<Id>(p.ids, i, p.n, experts);
            run = rank_tile(id);
        }
        __syncthreads();
        if (i < p.n) p.dest[i] = id < 0 ? -1 : s_next[id] + s_warp[warp * experts + id] + rank;
        if (t + 1 == tiles_per_block) break;
        __syncthreads();
        if (tid < experts) s_next[tid] += run;           // advance the experts past the tile
        clear_warps();
        __syncthreads();
    }
    if constexpr (kCluster) cluster_wait_acquire();
}

// --------------------------------------------------------------- dispatch ----
// Blocks [0, tokens): a token's row to its assignments' rows, read once.
// Blocks past them, one per expert: zeros into the group's padding rows.

// Eight columns of a row; kWhole: h % 8 == 0, so they are all inside (the other
// case's code and registers stay out of that instance).
template <bool kWhole>
__device__ __forceinline__ uint4 load8(const uint16_t *row, int c, int h)
{
    if (kWhole || c + 8 <= h) return *reinterpret_cast<const uint4 *>(row + c);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = c + i < h ? row[c + i] : 0u;
    return make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
}

template <bool kWhole>
__device__ __forceinline__ void store8(uint16_t *row, int c, int h, const uint4 &v)
{
    if (kWhole || c + 8 <= h) {
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
    const int d = p.dest[assignment];
    return d < p.rows ? d : -1;
}

// Zeros into a share of the padding rows (fewer than 128) of a group: item
// e * kPadSlices + j takes rows j, j + kPadSlices, ... of group e's.
constexpr int kPadSlices = 16;

template <bool kWhole>
__device__ __forceinline__ void zero_padding_rows(const MoeRowsParams &p, int item)
{
    const int e = item / kPadSlices;
    const int first = max(0, p.offsets[e] + p.counts[e]), end = min(p.offsets[e + 1], p.rows);
    for (int r = first + item % kPadSlices; r < end; r += kPadSlices)
        for (int c = threadIdx.x * 8; c < p.h; c += blockDim.x * 8)
            store8<kWhole>(p.out + (int64_t)r * p.ldo, c, p.h, make_uint4(0, 0, 0, 0));
}

// The rows of up to 8 assignments from `first` on, by lane (< 8; -1 past `count`).
__device__ __forceinline__ int rows_by_lane(const MoeRowsParams &p, int64_t first, int count)
{
    const int lane = threadIdx.x & 31;
    return lane < min(count, 8) ? row_of(p, first + lane) : -1;
}

template <bool kWhole>
__global__ void __launch_bounds__(256) moe_dispatch_kernel(const MoeRowsParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    if ((int)blockIdx.x >= p.tokens) {
        zero_padding_rows<kWhole>(p, blockIdx.x - p.tokens);
        return;
    }
    const int64_t first = (int64_t)blockIdx.x * p.topk;     // the token's assignments
    const uint16_t *x = p.x + (int64_t)blockIdx.x * p.ldx;
    for (int kb = 0; kb < p.topk; kb += 8) {
        const int mine = rows_by_lane(p, first + kb, p.topk - kb);
        for (int c0 = 0; c0 < p.h; c0 += blockDim.x * 8) {
            const int c = c0 + threadIdx.x * 8;
            const uint4 v = c < p.h ? load8<kWhole>(x, c, p.h) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int d = __shfl_sync(kFull, mine, k);
                if (d >= 0 && c < p.h) store8<kWhole>(p.out + (int64_t)d * p.ldo, c, p.h, v);
            }
        }
    }
}

// The same with the row quantized to NVFP4 on the way: one thread per
// 16-element block, four neighbours' scale codes stored as one word.
__global__ void __launch_bounds__(256) moe_dispatch_quant_kernel(const MoeRowsParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int64_t first = (int64_t)blockIdx.x * p.topk;     // the token's assignments
    const uint16_t *x = p.x + (int64_t)blockIdx.x * p.ldx;
    const float gs = *p.gs;
    const int steps = (p.nbp + blockDim.x - 1) / blockDim.x;
    for (int kb = 0; kb < p.topk; kb += 8) {                // (topk > 8 quantizes the row again per eight)
        const int mine = rows_by_lane(p, first + kb, p.topk - kb);
        for (int u = 0; u < steps; ++u) {
            const int blk = u * blockDim.x + threadIdx.x;
            const int k0 = blk * 16;
            const Raw16 raw = load16_coherent(x, k0, p.h);
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
            for (int k = 0; k < min(8, p.topk - kb); ++k) {
                const int r = __shfl_sync(kFull, mine, k);
                if (r < 0 || blk >= p.nb) continue;
                *reinterpret_cast<uint2 *>(p.q + (int64_t)r * (p.kp / 2) + k0 / 2) = q;
                if ((threadIdx.x & 3) == 0) *reinterpret_cast<uint32_t *>(p.sf + sf_offset(r, blk, p.nbp)) = word;
            }
        }
    }
}

// ---------------------------------------------------------------- combine ----
// A block takes its columns (eight per thread; blockIdx.y) of kT consecutive
// tokens at a time: the kT x kK rows of a step, up to eight 16-byte loads per
// thread, are requested together, with the next step's row numbers and weights
// behind them, so that one memory latency passes per step instead of two and a
// block start.  Small topk takes more tokens per step: with one row in flight
// per thread 16384 tokens of topk 1 moved 1.6 TB/s, with four 5.4 TB/s (the
// instance's bound of six blocks is 80 registers, 28 bytes spilled; 108 where
// h % 8 != 0).  topk > kK (= 8) goes round.
template <bool kWhole, int kK, int kT>
__global__ void __launch_bounds__(128, kK == 1 ? 6 : 8) moe_combine_kernel(const MoeRowsParams p)
{
    static_assert(kK * kT <= 8, "rows by lane");
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
    const bool here = c < p.h;
    // lane l < 8: assignment kb + l % kK of token t0 + l / kK
    auto row_at = [&](int t0, int kb) {
        const int t = t0 + lane / kK, k = kb + lane % kK;
        return lane < kK * kT && t < p.tokens && k < p.topk ? row_of(p, (int64_t)t * p.topk + k) : -1;
    };
    auto weight_at = [&](int row, int t0, int kb) {
        return row >= 0 && p.weights != nullptr ? p.weights[(int64_t)(t0 + lane / kK) * p.topk + kb + lane % kK] : 1.0f;
    };
    const int step = gridDim.x * kT;
    int mine = row_at(blockIdx.x * kT, 0);
    float my_w = weight_at(mine, blockIdx.x * kT, 0);
    for (int t0 = blockIdx.x * kT; t0 < p.tokens; t0 += step) {
        uint64_t acc[kT][4] = {};
        uint4 res[kT] = {};
        int next_mine = -1;
        float next_w = 1.0f;
        for (int kb = 0; kb < p.topk; kb += kK) {
            if (kb > 0) {
                mine = row_at(t0, kb);
                my_w = weight_at(mine, t0, kb);
            }
            uint4 v[kT][kK];
#pragma unroll
            for (int i = 0; i < kT * kK; ++i) {
                const int r = __shfl_sync(kFull, mine, i);
                v[i / kK][i % kK] =
                    r >= 0 && here ? load8<kWhole>(p.x + (int64_t)r * p.ldx, c, p.h) : make_uint4(0, 0, 0, 0);
            }
            if (kb == 0) {
                if (p.residual != nullptr && here)
#pragma unroll
                    for (int i = 0; i < kT; ++i)
                        if (t0 + i < p.tokens) res[i] = load8<kWhole>(p.residual + (int64_t)(t0 + i) * p.ldr, c, p.h);
                if (p.tokens - t0 > step) {
                    next_mine = row_at(t0 + step, 0);
                    next_w = weight_at(next_mine, t0 + step, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < kT * kK; ++i) {
                const float w = __shfl_sync(kFull, my_w, i); // (1 with zeros for a dropped assignment)
                const uint4 &u = v[i / kK][i % kK];
                uint64_t(&a)[4] = acc[i / kK];
                a[0] = fma2(bf16x2_to_f32x2(u.x), pack2(w, w), a[0]);
                a[1] = fma2(bf16x2_to_f32x2(u.y), pack2(w, w), a[1]);
                a[2] = fma2(bf16x2_to_f32x2(u.z), pack2(w, w), a[2]);
                a[3] = fma2(bf16x2_to_f32x2(u.w), pack2(w, w), a[3]);
            }
        }
        if (here)
#pragma unroll
            for (int i = 0; i < kT; ++i)
                if (t0 + i < p.tokens) {
                    if (p.residual != nullptr) add_residual8(acc[i], res[i]);
                    store8<kWhole>(p.out + (int64_t)(t0 + i) * p.ldo, c, p.h, bf16x8_of(acc[i]));
                }
        if (p.tokens - t0 <= step) break;                    // (t0 + step may pass 2^31: up to 2^31 tokens of topk 1)
        mine = next_mine;
        my_w = next_w;
    }
}

// Blocks as in moe_dispatch_kernel.  kK assignments at a time: their rows are
// requested together, each thread keeps kK partial dot products, and one
// reduction per kK (lanes, then warps, in a fixed order) ends them.  The
// instances for small topk hold fewer registers, so more tokens are in flight
// per SM.
template <bool kWhole, int kK>
__global__ void __launch_bounds__(256, kK == 8 ? 4 : kK == 4 ? 5 : 8) moe_combine_backward_kernel(const MoeRowsParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    if ((int)blockIdx.x >= p.tokens) {
        zero_padding_rows<kWhole>(p, blockIdx.x - p.tokens);
        return;
    }
    __shared__ float s_dot[8][kK];                       // [warp][assignment]
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *g = p.g + t * p.ldg;
    for (int kb = 0; kb < p.topk; kb += kK) {
        const int mine = lane < min(kK, p.topk - kb) ? row_of(p, t * p.topk + kb + lane) : -1;
        const float my_w = mine >= 0 ? p.weights[t * p.topk + kb + lane] : 0.0f;
        uint64_t dot[kK] = {};
        for (int c0 = 0; c0 < p.h; c0 += blockDim.x * 8) {
            const int c = c0 + threadIdx.x * 8;
            const bool here = c < p.h;
            uint4 v[kK];
#pragma unroll
            for (int k = 0; k < kK; ++k) {
                const int r = __shfl_sync(kFull, mine, k);
                v[k] = r >= 0 && here ? load8<kWhole>(p.x + (int64_t)r * p.ldx, c, p.h) : make_uint4(0, 0, 0, 0);
            }
            const uint4 gv = here ? load8<kWhole>(g, c, p.h) : make_uint4(0, 0, 0, 0);
            const uint64_t a[4] = {bf16x2_to_f32x2(gv.x), bf16x2_to_f32x2(gv.y), bf16x2_to_f32x2(gv.z),
                                   bf16x2_to_f32x2(gv.w)};
#pragma unroll
            for (int k = 0; k < kK; ++k) {
                const int r = __shfl_sync(kFull, mine, k);
                const float w = __shfl_sync(kFull, my_w, k);
                const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                uint64_t d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    dot[k] = fma2(a[i], bf16x2_to_f32x2(u[i]), dot[k]);
                    d[i] = mul2(a[i], pack2(w, w));
                }
                if (r >= 0 && here) store8<kWhole>(p.out + (int64_t)r * p.ldo, c, p.h, bf16x8_of(d));
            }
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            float lo, hi;
            unpack2(dot[k], lo, hi);
            float v = lo + hi;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
            if (lane == k) s_dot[warp][k] = v;
        }
        __syncthreads();
        if (threadIdx.x < kK && kb + (int)threadIdx.x < p.topk) {
            float sum = 0.0f;
            for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += s_dot[w][threadIdx.x];
            p.dw[t * p.topk + kb + threadIdx.x] = mine >= 0 ? sum : 0.0f;   // (lane k holds row k)
        }
        if (kb + kK < p.topk) __syncthreads();
    }
}

// Every kernel here is launched as a programmatic dependent and waits for the
// kernel before it (griddepcontrol.wait) before it reads or writes memory.
template <typename... Args>
cudaError_t launch_clusters(int cluster, void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                            Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args)
{
    return launch_clusters(1, kernel, grid, threads, smem, s, args...);
}

template <typename Id, bool kCluster>
cudaError_t launch_place(const MoeSortParams &p, int blocks, int per_block, cudaStream_t s)
{
    static int configured_device = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(moe_place_kernel<Id, kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             32 * kMoeMaxExperts * (int)sizeof(uint16_t));
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    return launch_clusters(kCluster ? blocks : 1, moe_place_kernel<Id, kCluster>, blocks, kMoeSortTile,
                           (size_t)32 * p.experts * sizeof(uint16_t), s, p, per_block);
}

template <typename Id>
cudaError_t launch_sort(const MoeSortParams &p, int num_sms, cudaStream_t s)
{
    const int tiles = p.n > 0 ? (p.n + kMoeSortTile - 1) / kMoeSortTile : 1;   // (no tokens: the offsets are still written)
    if (tiles <= kClusterTiles) return launch_place<Id, true>(p, tiles, 1, s);
    const int per_block = (tiles + num_sms - 1) / num_sms;
    const int blocks = (tiles + per_block - 1) / per_block;
    const cudaError_t e = launch_dependent(moe_count_kernel<Id>, blocks, kMoeSortTile, 0, s, p, per_block);
    return e != cudaSuccess ? e : launch_place<Id, false>(p, blocks, per_block, s);
}

// Threads for rows of h elements, eight per thread, and column parts of a row.
int row_threads(int h) { return h >= 2048 ? 256 : ((h + 7) / 8 + 31) / 32 * 32; }

}  // namespace

cudaError_t launch_moe_sort(const MoeSortParams &p, int num_sms, cudaStream_t s)
{
    return p.id_bytes == 8 ? launch_sort<int64_t>(p, num_sms, s) : launch_sort<int32_t>(p, num_sms, s);
}

cudaError_t launch_moe_dispatch(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    return launch_dependent(p.h % 8 == 0 ? moe_dispatch_kernel<true> : moe_dispatch_kernel<false>, (unsigned)(p.tokens + p.experts * kPadSlices), row_threads(p.h), 0,
                            s, p);
}

cudaError_t launch_moe_dispatch_quant(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    const int threads = p.nbp >= 256 ? 256 : (p.nbp + 31) / 32 * 32;
    return launch_dependent(moe_dispatch_quant_kernel, p.tokens, threads, 0, s, p);
}

namespace {

template <bool kWhole, int kK, int kT>
cudaError_t launch_combine(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    // 128 threads (fewer for short rows) of 64 registers at most: 1024 threads per SM
    // (topk 1: 80 registers and 768 threads; it has a block per step)
    const int threads = p.h >= 1024 ? 128 : ((p.h + 7) / 8 + 31) / 32 * 32, parts = (p.h + threads * 8 - 1) / (threads * 8);
    // (rounded down: one part of a step more than fits, and its blocks run alone at the end,
    // topk 8, 5120 columns, 6561 tokens: 119 us instead of 87)
    const int64_t resident = std::max<int64_t>(1, (int64_t)num_sms * (1024 / threads) / parts);
    const int64_t steps = (p.tokens + kT - 1) / kT;
    // Persistent blocks from six rounds on, but for topk 1.  A block per step / persistent,
    // us, at 2, 6, 12 and 27 rounds:
    //   topk 1, 5120 columns   7.4 / 8.4   22.0 / 24.8   42.8 / 48.8  106.7 / 107.7
    //   topk 2, 2048           5.4 / 5.0   15.1 / 14.3   34.0 / 29.8   76.1 / 62.9
    //   topk 8, 2048           8.4 / 8.0   21.7 / 22.2   43.1 / 40.8   92.7 / 87.2
    //   topk 8, 5120           8.6 / 8.9   22.2 / 22.5   41.5 / 41.0   94.1 / 86.8
    //   topk 3, 7168           4.3 / 4.4   10.9 / 11.1   21.9 / 21.5   46.9 / 45.0
    // Below six some sizes win by it and others lose, by a few percent either way.
    const int64_t blocks = kK == 1 || steps < 6 * resident ? steps : resident;
    return launch_dependent(moe_combine_kernel<kWhole, kK, kT>, dim3((unsigned)blocks, (unsigned)parts, 1), threads, 0, s,
                            p);
}

template <bool kWhole>
cudaError_t launch_combine_topk(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    return p.topk == 1   ? launch_combine<kWhole, 1, 4>(p, num_sms, s)
           : p.topk == 2 ? launch_combine<kWhole, 2, 2>(p, num_sms, s)
           : p.topk <= 4 ? launch_combine<kWhole, 4, 1>(p, num_sms, s)
                         : launch_combine<kWhole, 8, 1>(p, num_sms, s);
}

template <bool kWhole>
cudaError_t launch_combine_backward_topk(const MoeRowsParams &p, cudaStream_t s)
{
    void (*kernel)(MoeRowsParams) = p.topk == 1   ? moe_combine_backward_kernel<kWhole, 1>
                                    : p.topk == 2 ? moe_combine_backward_kernel<kWhole, 2>
                                    : p.topk <= 4 ? moe_combine_backward_kernel<kWhole, 4>
                                                  : moe_combine_backward_kernel<kWhole, 8>;
    return launch_dependent(kernel, (unsigned)(p.tokens + p.experts * kPadSlices), row_threads(p.h), 0, s, p);
}

}  // namespace

cudaError_t launch_moe_combine(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    return p.h % 8 == 0 ? launch_combine_topk<true>(p, num_sms, s) : launch_combine_topk<false>(p, num_sms, s);
}

cudaError_t launch_moe_combine_backward(const MoeRowsParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    return p.h % 8 == 0 ? launch_combine_backward_topk<true>(p, s) : launch_combine_backward_topk<false>(p, s);
}

}  // namespace nvfp4
