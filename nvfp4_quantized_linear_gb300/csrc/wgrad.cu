// Weight gradient of a linear from the 8-bit checkpoint of its input:
//   dw[j, c] = sum_r dy[r, j] * x[r, c],   dy bf16, x MXFP8,
// dense or per expert group, on the bf16 tensor cores of CTA pairs (tcgen05
// cta_group::2, kind::f16, fp32 accumulation in TMEM).
//
// An MXFP8 value is an E4M3 code times a power of two: four significant bits, so
// exact in bf16.  The kernel reads x at its 8 bits and widens it in shared memory
// on the way to the MMA.  The reduction runs over rows, along which both operands
// are strided, so both are MN-major: their tiles lie in shared memory as the rows
// lie in memory, 64 columns (128 bytes, 128-byte swizzle) a row.
//
// A tile is 256 (dy columns) x 256 (x columns); CTA r of the pair holds dy
// columns [128r, +128) and x columns [128r, +128) of it, 64 rows a stage.  Twenty-four
// warps per CTA:
//   warp 0       copies: two 64 x 64 boxes of dy, 64 x 128 codes and the 512-byte
//                scale tile of a stage
//   warp 1       allocates TMEM; in the leader one lane issues the pair's MMAs
//   warps 4..11  epilogue, two per TMEM lane quarter
//   warps 12..23 three groups, each widening every third stage's codes to bf16 (a ring
//                of its own: three slots, six stages of copies) and clearing the rows
//                past a group's last one in both operands (they may hold anything)
// Two accumulators of 256 columns fill TMEM, so a tile's epilogue runs under the
// next one's MMAs; a long sum, made of parts, takes both.
//
// 8192 rows, 28672 x 4096 in bf16: 1250 us, 1540 TFLOP/s (0.81 of cuBLAS's bf16 burst rate,
// 0.90 of its rate under the power cap).  Without the widening, its waits kept, 1165 us.
// What the steps before took: all widening warps on every stage 1850; a group of four for
// each of five stages 1400; its own ring and 8-byte pieces, 8 rows apart, 1205.
#include <algorithm>
#include <climits>
#include <mutex>

#include <cuda_bf16.h>

#include "block_launch.cuh"
#include "common.cuh"
#include "gemm_common.cuh"
#include "ptx.cuh"
#include "train_launch.cuh"

namespace nvfp4 {
namespace {

using namespace gemm_detail;

constexpr int kTile = 256;                               // per pair, both ways
constexpr int kHalf = 128;                               // per CTA
constexpr int kRows = 64;                                // of a stage
constexpr int kStages = 6;                               // of the copies
constexpr int kSlots = 3;                                // of widened x
constexpr uint32_t kBoxBytes = kRows * 128;              // 64 rows x 64 bf16 columns
constexpr uint32_t kOperandBytes = 2 * kBoxBytes;        // of one stage and CTA: 128 columns
constexpr uint32_t kCodeBytes = kRows * kHalf;
constexpr uint32_t kSfBytes = 512;
constexpr uint32_t kOffA = 0;
constexpr uint32_t kOffB = kOffA + kStages * kOperandBytes;
constexpr uint32_t kOffCodes = kOffB + kSlots * kOperandBytes;
constexpr uint32_t kOffSf = kOffCodes + kStages * kCodeBytes;
constexpr uint32_t kOffBar = kOffSf + kStages * kSfBytes;
constexpr uint32_t kOffTable = kOffBar + 256;            // groups by size
constexpr uint32_t kSmemBytes = kOffTable + 16 * kMoeMaxExperts + 1024;   // + alignment slack
constexpr uint32_t kTmemCols = 512;
constexpr int kThreads = 768;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8, kEpiCols = 128;      // columns of a tile per warp
// Warps of a group that widens every kSlots-th stage: a group for every slot, so that
// each group waits for every use of its barriers in turn.  (Groups that take turns on a
// stage do not: copies land out of order, and a parity cannot tell a use from the one two
// back.)
constexpr int kConvWarp0 = 12, kConvWarps = 4;
constexpr int kPieces = kRows * kHalf / 8 / (kConvWarps * 32);    // 8-byte pieces of codes per thread and stage
static_assert((kConvWarp0 + kConvWarps * kSlots) * 32 == kThreads, "warps");
static_assert(kStages % kSlots == 0, "a group's stages are its own");
static_assert(kPieces == 8 && kRows == 64, "a thread's rows are eight apart");
constexpr uint16_t kBothCtas = 0x3;

// Rows of one sum on the tensor cores, whose accumulator is truncated, not rounded, at every step
// of 16 rows: a sum of one sign falls short by 2.1e-6 of itself after 2048 rows, 1.2e-5 after
// 8192, 1.9e-4 after 65536 (of both signs by 6e-7, 3.5e-6).  The parts of a longer sum are added in the other accumulator, in fp32 and rounded to nearest, which holds the
// tensor cores up for a drain a part: 8192 rows, 28672 x 4096 in bf16 1250 us with parts of 8192
// rows, 1265 with 4096, 1315 with 2048, 1397 with 1024.  A bf16 gradient is rounded to 2^-9 and takes
// the longest; an fp32 one's parts cost no more than its stores (16384 rows, 8192 x 4096: 744 us, added to
// dw in memory 752).
constexpr int kPartRows = 2048, kPartRowsBf16 = 8192;

static_assert(kSmemBytes <= 232448, "shared memory budget");

// Descriptor of an MN-major operand: 64-column boxes of kBoxBytes (leading byte
// offset), inside a box groups of eight rows 1024 bytes apart (stride byte offset).
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kBoxBytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// bf16 x bf16 with both operands MN-major (bits 15 and 16).
constexpr uint32_t kIdesc = idesc_bf16(kTile, kTile) | (1u << 15) | (1u << 16);

__device__ __forceinline__ void tc_mma_pair_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// v += 32 columns of TMEM.
__device__ __forceinline__ void tmem_add_32cols(uint32_t taddr, uint32_t (&v)[32])
{
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        uint32_t u[16];
        tmem_ld_16cols(taddr + h, u);
        tmem_ld_wait_regs(u);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[h + i] = __float_as_uint(__uint_as_float(u[i]) + __uint_as_float(v[h + i]));
    }
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// A tile of the walk: its group's rows and its first dy and x columns.
struct WTile {
    int first, rows;                                     // rows [first, first + rows)
    int group, n0, k0;
};

// Tile number `at` of the walk; table: {group, first row, rows} of the groups by
// descending size.
__device__ __forceinline__ WTile tile_of(const WgradParams &p, int at, const int4 *table)
{
    const int per_group = p.num_n_blk * p.num_k_blk;
    const int g = at / per_group;
    const Tile t = tile_coord(at - g * per_group, p.num_n_blk, p.num_k_blk, 5);
    WTile w = {0, p.m, g, t.mb * kTile, t.nb * kTile};
    if (p.offsets != nullptr) {
        const int4 e = table[g];
        w.group = e.x;
        w.first = e.y;
        w.rows = e.z;
    } else {                                             // a range of the rows
        w.first = min(g * p.span, p.m);
        w.rows = min(p.span, p.m - w.first);
    }
    return w;
}

// The tiles of a pair: rounds over the pairs, every other one backwards, so that with
// the groups by descending size the pairs' shares of the rows are about even
// (in plain turns the busiest pair of the routed case has 10 to 45 % more
// rows than the mean one, this way 3 to 5 %).
struct Walk {
    int pair, pairs, tiles, round;
    __device__ __forceinline__ int first() { round = 0; return pair; }
    __device__ __forceinline__ int next()
    {
        ++round;
        return round * pairs + (round & 1 ? pairs - 1 - pair : pair);
    }
};

// The block's threads: the groups by size (equal ones by number) into the table.
// `counts`: shared memory for num_groups (rounded up to 4) words.
__device__ __forceinline__ void order_groups(const WgradParams &p, int4 *table, int32_t *counts)
{
    const int padded = (p.num_groups + 3) / 4 * 4;
    for (int g = threadIdx.x; g < padded; g += kThreads) counts[g] = g < p.num_groups ? p.counts[g] : INT_MIN;
    __syncthreads();
    for (int g = threadIdx.x; g < p.num_groups; g += kThreads) {
        const int mine = counts[g], first = min(max(p.offsets[g], 0), p.m);
        int rank = 0;
        for (int h = 0; h < padded; h += 4) {
            const int4 c = *reinterpret_cast<const int4 *>(counts + h);
            rank += (c.x > mine || (c.x == mine && h < g)) + (c.y > mine || (c.y == mine && h + 1 < g)) +
                    (c.z > mine || (c.z == mine && h + 2 < g)) + (c.w > mine || (c.w == mine && h + 3 < g));
        }
        table[rank] = make_int4(g, first, min(max(mine, 0), p.m - first), 0);
    }
    __syncthreads();
}

// Four codes times a power of two as two bf16 pairs.  A code's exponent and mantissa
// moved to bf16's places are its value times 2^-120 (the difference of the exponent
// biases), subnormals included.
__device__ __forceinline__ uint32_t widen2(uint32_t pair, uint32_t factor)
{
    return mul_bf16x2((pair & 0x80008000u) | ((pair >> 4) & 0x07F007F0u), factor);
}

__device__ __forceinline__ void widen4(uint32_t w, uint32_t factor, uint32_t &lo, uint32_t &hi)
{
    lo = widen2(__byte_perm(w, 0, 0x1404), factor);
    hi = widen2(__byte_perm(w, 0, 0x3424), factor);
}

// A top bit of a byte if one of the four codes is E4M3's NaN (0x7F with either sign), which one
// more takes over its sign bit.  (A carry out of 0xFF may set others: two instructions a word
// for a look that finds nothing nearly always, 1 to 2 % of the time.)
__device__ __forceinline__ uint32_t maybe_nan(uint32_t w) { return (w + 0x01010101u) ^ w; }

// NaN for those codes in the four values of widen4.
__device__ __forceinline__ void put_nan(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t n = (w & 0x7F7F7F7Fu) + 0x01010101u;
    lo |= (n & 0x80u ? 0x7FC0u : 0) | (n & 0x8000u ? 0x7FC00000u : 0);
    hi |= (n & 0x800000u ? 0x7FC0u : 0) | (n & 0x80000000u ? 0x7FC00000u : 0);
}

// Adds four floats to memory without waiting for them (rounded to nearest, subnormals
// flushed).
__device__ __forceinline__ void red_add_v4(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(__uint_as_float(a)), "f"(__uint_as_float(b)),
                 "f"(__uint_as_float(c)), "f"(__uint_as_float(d))
                 : "memory");
}

// Transposes units of kUnit words among groups of kWords / kUnit neighbouring lanes: lane j of a
// group has its row's units before, and unit j of the group's rows after, row i's at v[i * kUnit].
template <int kUnit, int kWords>
__device__ __forceinline__ void transpose_units(uint32_t (&v)[kWords], int lane)
{
    constexpr int kLanes = kWords / kUnit;
#pragma unroll
    for (int b = 1; b < kLanes; b <<= 1) {
        const bool high = lane & b;
#pragma unroll
        for (int i = 0; i < kLanes; ++i) {
            if (i & b) continue;
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                uint32_t &lo = v[i * kUnit + j], &hi = v[(i | b) * kUnit + j];
                const uint32_t got = __shfl_xor_sync(~0u, high ? lo : hi, b);
                if (high) lo = got;
                else hi = got;
            }
        }
    }
}

// 32 bytes of a row, as one store where they are a sector.
__device__ __forceinline__ void store_32_bytes(void *o, const uint32_t *v)
{
    if ((reinterpret_cast<uintptr_t>(o) & 31) == 0) {
        st_global_v8(o, *reinterpret_cast<const uint32_t(*)[8]>(v));
    } else {
        static_cast<uint4 *>(o)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4 *>(o)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// A warp's 32 rows x 32 whole columns (a row per lane; o: the first row, `ld` elements apart; `rows` of
// them are there) to memory, pairs of lanes side by side: a store instruction then writes 64 bytes
// of 16 lines instead of 32 of 32, and the stores stand less in the way of the widening's
// accesses to shared memory.  64 rows, 28672 x 4096: a row per lane 105 us in fp32 and 70 in bf16, this
// way 83 and 61 (whole lines of fp32, twice the shuffles: 90).
__device__ __forceinline__ void store_rows_f32(float *o, int64_t ld, int rows, uint32_t (&v)[32], int lane)
{
    transpose_units<16>(v, lane);
    o += (lane & ~1) * ld + (lane & 1) * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i, o += ld) {
        if ((lane & ~1) + i >= rows) continue;
        store_32_bytes(o, v + 16 * i);
        store_32_bytes(o + 8, v + 16 * i + 8);
    }
}

// Added to memory: whole lines (8192 routed tokens' gradients, parts of 1024 rows: 224 us, a row per lane 252).
__device__ __forceinline__ void add_rows_f32(float *o, int64_t ld, int rows, uint32_t (&v)[32], int lane)
{
    transpose_units<4>(v, lane);
    o += (lane & ~7) * ld + (lane & 7) * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i, o += ld)
        if ((lane & ~7) + i < rows) red_add_v4(o, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// The same in bf16.
__device__ __forceinline__ void store_rows_bf16(uint16_t *o, int64_t ld, int rows, const uint32_t (&v)[32], int lane)
{
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = bf16x2_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
    transpose_units<8>(w, lane);
    o += (lane & ~1) * ld + (lane & 1) * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i, o += ld)
        if ((lane & ~1) + i < rows) store_32_bytes(o, w + 8 * i);
}

// The first `cols` (< 32) of 32 columns of one thread's row: where a row ends inside them.
__device__ __forceinline__ void store_row_end(const WgradParams &p, int64_t at, int cols, const uint32_t (&v)[32], bool add)
{
    const bool f32 = p.type == kTypeF32;
    float *o = static_cast<float *>(p.dw) + at;
    uint16_t *h = static_cast<uint16_t *>(p.dw) + at;
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
        if (j >= cols) break;
        if (j + 8 <= cols && !f32) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = bf16x2_rn(__uint_as_float(v[j + 2 * i]), __uint_as_float(v[j + 2 * i + 1]));
            *reinterpret_cast<uint4 *>(h + j) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if (j + 8 <= cols && !add) {
            *reinterpret_cast<uint4 *>(o + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            *reinterpret_cast<uint4 *>(o + j + 4) = make_uint4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (j + i >= cols) break;
                if (f32) o[j + i] = __uint_as_float(v[j + i]) + (add ? o[j + i] : 0.0f);
                else h[j + i] = (uint16_t)bf16_bits_rn(__uint_as_float(v[j + i]));
            }
        }
    }
}

// Largest scale code whose factor 2^(code - 127 + 120) bf16 holds.
constexpr uint32_t kOneFactor = 134;

__global__ void __launch_bounds__(kThreads, 1)
    wgrad_pair_kernel(const __grid_constant__ CUtensorMap tmDy, const __grid_constant__ CUtensorMap tmCodes,
                      const WgradParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar);    // this CTA's copies of the stage landed
    uint64_t *ready = full + kStages;                                  // (leader) both CTAs widened into the slot
    uint64_t *empty = ready + kSlots;                                  // the pair's MMAs released the stage and its slot
    uint64_t *tmem_full = empty + kStages;                             // [2] accumulator complete
    uint64_t *tmem_empty = tmem_full + 2;                              // [2] (leader) both CTAs drained it
    uint64_t *mma_done = tmem_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    int4 *const table = reinterpret_cast<int4 *>(smem + kOffTable);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kSlots; ++s) mbar_init(&ready[s], 2 * kConvWarps);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tmem_full[b], 1);
            mbar_init(&tmem_empty[b], 2 * kEpiWarps);
        }
        mbar_init(mma_done, 1);
        fence_mbarrier_init();
        prefetch_tensormap(&tmDy);
        prefetch_tensormap(&tmCodes);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncwarp();
    cluster_sync_all();
    tc_fence_after_sync();
    griddep_launch_dependents();
    griddep_wait();
    if (p.offsets != nullptr) order_groups(p, table, reinterpret_cast<int32_t *>(smem + kOffB));   // (not in use yet)

    const uint32_t tmem = role_tmem(tmem_slot);
    const uint32_t rank = cluster_ctarank();
    Walk walk = {(int)(blockIdx.x >> 1), (int)(gridDim.x >> 1), p.num_groups * p.num_n_blk * p.num_k_blk, 0};

    if (warp >= kConvWarp0) {
        // ------------------------------------------------------- widening --
        // A thread widens eight codes of each of its eight rows, eight rows apart: 16 lanes
        // a row, so that both the 8-byte loads and the 16-byte stores hit every bank once,
        // and rows that are alike modulo 8 have one place in the swizzle.
        const int group = (warp - kConvWarp0) / kConvWarps;
        const int row0 = ((warp - kConvWarp0) % kConvWarps) * 2 + (lane >> 4);
        const int col8 = lane & 15;                      // 8-column piece
        const uint32_t leader_ready = mapa_shared(&ready[group], 0);
        const uint32_t in_codes = smem_u32(smem + kOffCodes) + row0 * kHalf + col8 * 8;
        const uint32_t in_sf = smem_u32(smem + kOffSf) + row0 * 16 + (col8 >> 2);
        const uint32_t a_row = smem_u32(smem + kOffA) + (col8 >> 3) * kBoxBytes + row0 * 128 + (col8 & 7) * 16;
        const uint32_t out = smem_u32(smem + kOffB) + group * kOperandBytes + (col8 >> 3) * kBoxBytes + row0 * 128 +
                             (((col8 & 7) ^ row0) << 4);
        int next = group, stage = group;                 // the group's next stage, of the tile and of the ring
        int before = -1;                                 // the stage whose MMAs read the slot last
        uint32_t phase = 0, before_phase = 0;
        bool ok = true;
        for (int tile = walk.first(); tile < walk.tiles && ok; tile = walk.next()) {
            const WTile t = tile_of(p, tile, table);
            const int num_ks = (t.rows + kRows - 1) / kRows;
            for (; next < num_ks; next += kSlots) {
                ok = __all_sync(~0u, mbar_wait(&full[stage], phase, p.err_flag, kErrTimeout, p.wait_ns));
                if (!ok) break;
                const uint32_t band_half = (uint32_t)next & 1u;
                uint2 w[kPieces];
                uint32_t code[kPieces], top = 0, nans = 0;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    w[i] = ld_shared_v2(in_codes + stage * kCodeBytes + i * 8 * kHalf);
                    code[i] = ld_shared_u8(in_sf + stage * kSfBytes + band_half * 8 + (i & 3) * 128 + (i >> 2) * 4);
                    top = max(top, code[i]);
                    nans |= maybe_nan(w[i].x);
                    nans |= maybe_nan(w[i].y);
                }
                if (before >= 0) {
                    ok = __all_sync(~0u, mbar_wait(&empty[before], before_phase, p.err_flag, kErrTimeout, p.wait_ns));
                    if (!ok) break;
                }
                if (!__any_sync(~0u, top > kOneFactor || (nans & 0x80808080u) != 0)) {
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const uint32_t f = code[i] * 0x00800080u + 120 * 0x00800080u;
                        uint32_t v[4];
                        widen4(w[i].x, f, v[0], v[1]);
                        widen4(w[i].y, f, v[2], v[3]);
                        st_shared_v4(out + i * 1024, v[0], v[1], v[2], v[3]);
                    }
                } else {
                    // the part of a factor past bf16's range as a second one, NaN codes and blocks
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const uint32_t c1 = min(code[i], kOneFactor);
                        const uint32_t f1 = code[i] == 255 ? 0x7FC07FC0u : (c1 + 120) * 0x00800080u;
                        const uint32_t f2 = (127 + code[i] - c1) * 0x00800080u;
                        uint32_t v[4];
                        widen4(w[i].x, f1, v[0], v[1]);
                        widen4(w[i].y, f1, v[2], v[3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = mul_bf16x2(v[j], f2);
                        put_nan(w[i].x, v[0], v[1]);
                        put_nan(w[i].y, v[2], v[3]);
                        st_shared_v4(out + i * 1024, v[0], v[1], v[2], v[3]);
                    }
                }
                const int valid = t.rows - next * kRows;
                if (valid < kRows)                       // rows of nobody: zeros, in dy's boxes too
#pragma unroll
                    for (int i = 0; i < kPieces; ++i)
                        if (row0 + 8 * i >= valid) {
                            st_shared_v4(out + i * 1024, 0, 0, 0, 0);
                            st_shared_v4(a_row + stage * kOperandBytes + i * 1024, 0, 0, 0, 0);
                        }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(&ready[group]);
                    else mbar_arrive_remote(leader_ready);
                }
                before = stage;
                before_phase = phase;
                stage += kSlots;
                if (stage >= kStages) { stage -= kStages; phase ^= 1; }
            }
            next -= num_ks;
        }
    } else if (warp >= kEpiWarp0) {
        // ------------------------------------------------------- epilogue --
        const int q = warp & 3;
        const int col0 = (warp - kEpiWarp0) / 4 * kEpiCols;
        const uint32_t leader_empty = mapa_shared(tmem_empty, 0);
        uint32_t phase[2] = {0, 0};
        int buf = 0;
        bool ok = true;
        for (int tile = walk.first(); tile < walk.tiles && ok; tile = walk.next()) {
            const WTile t = tile_of(p, tile, table);
            if (t.rows == 0 && p.accumulate) continue;
            const int n0 = t.n0 + (int)rank * kHalf + q * 32;
            const int64_t plane = ((int64_t)t.group * p.n + n0) * p.ldw;
            // (held: the sum of the parts so far stays in accumulator buf, the next ones come in the other)
            const bool held = t.rows > p.part_rows;
            for (int left = t.rows; ok; left -= p.part_rows) {
                const bool begun = left < t.rows, last = left <= p.part_rows;
                const int part = held && begun ? buf ^ 1 : buf;
                const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + part * kTile + col0;
                const uint32_t sum = tmem + ((uint32_t)(q * 32) << 16) + buf * kTile + col0;
                if (t.rows > 0) {
                    ok = __all_sync(~0u, mbar_wait(&tmem_full[part], phase[part], p.err_flag, kErrTimeout, p.wait_ns));
                    if (!ok) break;
                    phase[part] ^= 1;
                    tc_fence_after_sync();
                }
                if (held && !begun) continue;
#pragma unroll 1
                for (int ch = 0; ch < kEpiCols / 32; ++ch) {
                    const int c = t.k0 + col0 + ch * 32;
                    if (c >= p.dw_cols || n0 >= p.n) break;
                    uint32_t v[32];
                    if (t.rows > 0) {
                        tmem_ld_32cols(acc + ch * 32, v);
                        tmem_ld_wait_regs(v);
                        if (held) {
                            tmem_add_32cols(sum + ch * 32, v);
                            if (!last) {
                                tmem_st_32cols(sum + ch * 32, v);
                                continue;
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0;
                    }
                    const int rows = p.n - n0;
                    const int64_t at = plane + c;
                    if (c + 32 > p.dw_cols) {
                        if (lane < rows) store_row_end(p, at + lane * p.ldw, p.dw_cols - c, v, p.accumulate);
                    } else if (p.type != kTypeF32) {
                        store_rows_bf16(static_cast<uint16_t *>(p.dw) + at, p.ldw, rows, v, lane);
                    } else if (p.accumulate) {
                        add_rows_f32(static_cast<float *>(p.dw) + at, p.ldw, rows, v, lane);
                    } else {
                        store_rows_f32(static_cast<float *>(p.dw) + at, p.ldw, rows, v, lane);
                    }
                    __syncwarp();
                }
                if (t.rows > 0) {
                    if (held) tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        for (int b = 0; b < 2; ++b) {
                            if (b != part && !(held && last)) continue;
                            if (rank == 0) mbar_arrive(&tmem_empty[b]);
                            else mbar_arrive_remote(leader_empty + b * (uint32_t)sizeof(uint64_t));
                        }
                    }
                    if (!held) buf ^= 1;
                }
                if (last) break;
            }
        }
    } else if (warp == 0 && lane == 0) {
        // --------------------------------------------------------- copies --
        const uint64_t pol = l2_policy_evict_last();
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_phase = 0;
        bool ok = true;
        for (int tile = walk.first(); tile < walk.tiles && ok; tile = walk.next()) {
            const WTile t = tile_of(p, tile, table);
            const int n = t.n0 + (int)rank * kHalf, k = t.k0 + (int)rank * kHalf;
            const bool sf_here = k < p.sf_tiles * 128;
            for (int r0 = 0; r0 < t.rows; r0 += kRows) {
                if (!mbar_wait(&empty[stage], phase ^ 1, p.err_flag, kErrTimeout, p.wait_ns)) {
                    ok = false;
                    break;
                }
                const int row = t.first + r0;
                // (boxes past the last row or column are zero-filled and count their bytes)
                mbar_arrive_expect_tx(&full[stage], kOperandBytes + kCodeBytes + (sf_here ? kSfBytes : 0));
                tma_load_2d(smem + kOffCodes + stage * kCodeBytes, &tmCodes, &full[stage], k, row, pol);
                if (sf_here)
                    bulk_load(smem + kOffSf + stage * kSfBytes,
                              p.sf + ((int64_t)(row >> 7) * p.sf_tiles + (k >> 7)) * kSfBytes, kSfBytes, &full[stage], pol);
                tma_load_2d(smem + kOffA + stage * kOperandBytes, &tmDy, &full[stage], n, row, pol);
                tma_load_2d(smem + kOffA + stage * kOperandBytes + kBoxBytes, &tmDy, &full[stage], n + 64, row, pol);
                issued |= 1u << stage;
                issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == kStages) { stage = 0; phase ^= 1; }
            }
        }
        for (int s = 0; s < kStages; ++s)                // nothing in flight when the CTA ends
            if (issued & (1u << s)) mbar_wait(&full[s], (issued_phase >> s) & 1u, p.err_flag, kErrTimeout, p.wait_ns);
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ MMA --
        const bool issuer = elect_one();
        const uint32_t a_base = smem_u32(smem + kOffA), b_base = smem_u32(smem + kOffB);
        int stage = 0, slot = 0, buf = 0;
        uint32_t phase = 0, acc_phase[2] = {0, 0};
        bool ok = true;
        for (int tile = walk.first(); tile < walk.tiles && ok; tile = walk.next()) {
            const WTile t = tile_of(p, tile, table);
            const int first = buf;
            const bool held = t.rows > p.part_rows;      // (as in the epilogue)
            for (int left = t.rows; left > 0 && ok; left -= p.part_rows) {
                if (held && left < t.rows) buf = first ^ 1;
                ok = __all_sync(~0u, mbar_wait(&tmem_empty[buf], acc_phase[buf] ^ 1, p.err_flag, kErrTimeout, p.wait_ns));
                if (!ok) break;
                tc_fence_after_sync();
                const int rows = min(p.part_rows, left);
                for (int r0 = 0; r0 < rows; r0 += kRows) {
                    ok = __all_sync(~0u, mbar_wait(&ready[slot], phase, p.err_flag, kErrTimeout, p.wait_ns));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const int steps = min(kRows / 16, (rows - r0 + 15) / 16);
                    const uint64_t ad = desc_mn_sw128(a_base + stage * kOperandBytes);
                    const uint64_t bd = desc_mn_sw128(b_base + slot * kOperandBytes);
                    if (issuer) {
                        for (int kk = 0; kk < steps; ++kk)   // 16 rows of 128 bytes
                            tc_mma_pair_bf16(tmem + buf * kTile, ad + kk * (2048 >> 4), bd + kk * (2048 >> 4), kIdesc,
                                             (r0 | kk) != 0);
                        tc_commit_pair_multicast(&empty[stage], kBothCtas);
                    }
                    if (++stage == kStages) stage = 0;
                    if (++slot == kSlots) { slot = 0; phase ^= 1; }
                }
                if (!ok) break;
                if (issuer) tc_commit_pair_multicast(&tmem_full[buf], kBothCtas);
                __syncwarp();
                acc_phase[buf] ^= 1;
                buf ^= 1;
            }
            if (held) buf = first;
        }
        if (issuer) tc_commit_pair(mma_done);
        __syncwarp();
        mbar_wait(mma_done, 0, p.err_flag, kErrTimeout, p.wait_ns);
    }

    tc_fence_before_sync();
    __syncwarp();
    cluster_sync_all();                 // no peer access to this CTA's smem or TMEM after this point
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

// dw = (dw +) the ranges' sums, in their order; a thread takes eight columns.
__global__ void __launch_bounds__(256) wgrad_sum_kernel(const WgradParams p, const float *parts, int splits, int64_t part, int cols)
{
    griddep_launch_dependents();
    griddep_wait();
    const int64_t pieces = (int64_t)p.n * (cols / 8);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / (cols / 8);
        const int c = (int)(i - row * (cols / 8)) * 8;
        const float *src = parts + row * cols + c;
        const int left = min(8, p.k - c);
        float v[8] = {};
        float *o32 = static_cast<float *>(p.dw) + row * p.ldw + c;
        if (p.accumulate)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < left) v[j] = o32[j];
        for (int s = 0; s < splits; ++s) {
            const float4 a = *reinterpret_cast<const float4 *>(src + s * part);
            const float4 b = *reinterpret_cast<const float4 *>(src + s * part + 4);
            const float u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += u[j];
        }
        if (p.type == kTypeF32) {
            if (left == 8) {
                *reinterpret_cast<float4 *>(o32) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(o32 + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < left) o32[j] = v[j];
            }
        } else {
            uint16_t *o = static_cast<uint16_t *>(p.dw) + row * p.ldw + c;
            if (left == 8) {
                *reinterpret_cast<uint4 *>(o) = make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]),
                                                           bf16x2_rn(v[6], v[7]));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < left) o[j] = (uint16_t)bf16_bits_rn(v[j]);
            }
        }
    }
}

bool make_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t cols, uint64_t rows, uint64_t row_bytes,
              uint32_t box_cols, CUtensorMapSwizzle swizzle)
{
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {box_cols, kRows};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

namespace {

// Row ranges of one weight of few tiles: as many as keep the pairs of a GPU of 152 SMs
// busy in one round, of 512 rows at least.
constexpr int kPairs = 76, kMinSpan = 512;

int wgrad_splits(int64_t m, int64_t n, int64_t k)
{
    const int64_t tiles = ((n + kTile - 1) / kTile) * ((k + kTile - 1) / kTile);
    return (int)std::max<int64_t>(1, std::min<int64_t>({kPairs / tiles, 8, m / kMinSpan}));
}

int64_t padded_cols(int64_t k) { return (k + 7) / 8 * 8; }

}  // namespace

size_t wgrad_workspace_bytes(int64_t m, int64_t n, int64_t k, int groups)
{
    const int splits = groups > 0 ? 1 : wgrad_splits(m, n, k);
    return splits > 1 ? (size_t)splits * n * padded_cols(k) * sizeof(float) : 0;
}

cudaError_t launch_wgrad(const WgradParams &p_in, const uint16_t *dy, int64_t ldd, const uint8_t *q, void *workspace,
                         int num_sms, cudaStream_t s, const char **why)
{
    static std::mutex mutex;
    static int configured_device = -1;
    static int known_pairs = 0;
    int dev = 0, max_pairs = 0;
    cudaGetDevice(&dev);
    std::unique_lock<std::mutex> lock(mutex);
    if (configured_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(wgrad_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t probe = {};
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        probe.gridDim = dim3(2 * (num_sms / 2), 1, 1);
        probe.blockDim = dim3(kThreads, 1, 1);
        probe.dynamicSmemBytes = kSmemBytes;
        probe.attrs = &attr;
        probe.numAttrs = 1;
        int clusters = 0;
        e = cudaOccupancyMaxActiveClusters(&clusters, wgrad_pair_kernel, &probe);
        if (e != cudaSuccess || clusters < 1) {
            cudaGetLastError();
            clusters = num_sms / 2;
        }
        known_pairs = clusters;
        configured_device = dev;
    }
    max_pairs = known_pairs;
    lock.unlock();
    WgradParams p = p_in;
    p.num_n_blk = (p.n + kTile - 1) / kTile;
    p.num_k_blk = (p.k + kTile - 1) / kTile;
    p.dw_cols = p.k;
    p.span = p.m;
    const int splits = p.offsets != nullptr ? 1 : wgrad_splits(p.m, p.n, p.k);
    if (splits > 1) {                                    // fp32 sums of the ranges, added by a second kernel
        p.span = ((p.m + splits - 1) / splits + 127) / 128 * 128;
        p.num_groups = splits;
        p.type = kTypeF32;
        p.accumulate = 0;
        p.dw = workspace;
        p.ldw = p.dw_cols = (int32_t)padded_cols(p.k);
    }
    p.part_rows = p.type == kTypeF32 ? kPartRows : kPartRowsBf16;
    // (no rows: the maps are not read)
    const void *dy_base = p.m > 0 ? static_cast<const void *>(dy) : p.dw, *q_base = p.m > 0 ? q : p.dw;
    const uint64_t rows = p.m > 0 ? (uint64_t)p.m : 1;
    CUtensorMap tmDy, tmCodes;
    if (!make_map(&tmDy, CU_TENSOR_MAP_DATA_TYPE_UINT16, dy_base, (uint64_t)p.n, rows,
                  p.m > 0 ? (uint64_t)ldd * 2 : ((uint64_t)p.n * 2 + 15) / 16 * 16, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&tmCodes, CU_TENSOR_MAP_DATA_TYPE_UINT8, q_base, (uint64_t)p.kp, rows, (uint64_t)p.kp, kHalf,
                  CU_TENSOR_MAP_SWIZZLE_NONE)) {
        *why = "cuTensorMapEncodeTiled failed for an operand of the weight gradient";
        return cudaErrorInvalidValue;
    }
    const int tiles = p.num_groups * p.num_n_blk * p.num_k_blk;
    const int pairs = std::min(tiles, max_pairs);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.x = 2;
    attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
    attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, wgrad_pair_kernel, tmDy, tmCodes, p);
    if (splits == 1 || e != cudaSuccess) return e;
    const int cols = p.dw_cols;
    const int64_t pieces = (int64_t)p.n * (cols / 8);
    cfg.gridDim = dim3((unsigned)std::min<int64_t>((pieces + 255) / 256, (int64_t)num_sms * 8));
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    cfg.attrs = attrs + 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, wgrad_sum_kernel, p_in, static_cast<const float *>(workspace), splits,
                              (int64_t)p.n * cols, cols);
}

}  // namespace nvfp4
