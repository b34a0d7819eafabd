// Pieces shared by the tensor-core kernels (the two GEMMs and the transform
// quantizer): tile order, tensor-map builders.
#pragma once

#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "epilogue.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace gemm_detail {

struct Tile {
    int mb, nb;
};

// 512-byte scale tiles (128 rows x 4 scale columns) per 128-row band in one
// 256-element K stage: NVFP4 has a scale per 16 elements (4 tiles), MXFP4 one
// per 32 (2 tiles).
template <bool kMx>
constexpr int kSfTilesPerStage = kMx ? 2 : 4;

// Tiles are walked column by column (row band fastest) inside groups of
// `group` row bands (at most): the CTAs resident at one time work on a few
// weight column bands, so each weight tile is streamed from DRAM about once
// and shared by the row bands through L2, while the group's activation rows
// stay resident in L2 across columns.  Both GEMM kernels use groups of 8192
// activation rows (64 bands of 128 rows, or 32 pair tiles of 256 rows): on the
// Qwen gate_up shape (M = 16384, K = 5120) the CTA-pair kernel measured
// 1278 us with 32-tile groups against 1327 us with 64 and 1311 / 1385 us with
// 16 / 8.
__device__ __forceinline__ Tile tile_coord(int tile, int num_m, int num_n, int group = 64)
{
    const int G = num_m < group ? num_m : group;
    const int per_group = G * num_n;
    const int grp = tile / per_group;
    const int first_m = grp * G;
    const int gm = min(G, num_m - first_m);
    const int within = tile - grp * per_group;
    return {first_m + within % gm, within / gm};
}

__device__ __forceinline__ uint32_t bf16_bits_rn(float f)
{
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f));
}


// An opaque copy.  The roles of the GEMM kernels read what they need (lane, tile
// counts, TMEM address) through it at their start: a value computed once before
// the roles part is one variable in all of them, and where the epilogue's
// registers run out it is spilled in all; the MMA and copy loops then reload it
// from memory in every stage (the CTA-pair kernel with a residual measured 162 us
// at 8192 x 14336 x 4096 against 138 us without those spills).
__device__ __forceinline__ int role_value(int v)
{
    asm volatile("" : "+r"(v));
    return v;
}

__device__ __forceinline__ uint32_t role_tmem(const uint32_t *tmem_slot)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(tmem_slot)));
    return v;
}

// The TMA clips an output row at 16-byte granularity: the output maps cover the
// first out_cols / 8 * 8 columns, and the up to seven columns past them are
// written by the row's thread from its staged 16-byte piece `v`.
__host__ __device__ constexpr int tma_cols(int out_cols) { return out_cols & ~7; }

__device__ __forceinline__ void store_tail_columns(const GemmParams &p, int64_t row, const uint4 &v)
{
    const int c0 = tma_cols(p.out_cols), n = p.out_cols - c0;
    uint16_t *o = p.out + row * p.ldo + c0;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) o[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
}

// One warp stores its staged 32-row x 64-column output chunk (128-byte rows with
// the TMA's 128-byte swizzle; kTail: the output's last columns may end inside 16
// bytes).
template <bool kTail>
__device__ __forceinline__ void store_chunk(const GemmParams &p, const CUtensorMap *map, uint32_t stage, int col, int row,
                                            int lane, uint64_t policy)
{
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0 && (!kTail || col < tma_cols(p.out_cols))) {
        tma_store_2d(map, stage, col, row, policy);
        bulk_commit_group();
    }
    if (kTail && (p.out_cols & 7) != 0) {           // uniform: the chunk that holds the last columns
        const int piece = (tma_cols(p.out_cols) - col) >> 3;
        if (piece >= 0 && piece < 8 && row + lane < p.m)
            store_tail_columns(p, row + lane, ld_shared_v4(stage + lane * 128 + ((piece ^ (lane & 7)) << 4)));
    }
}

// The epilogue variant a launch needs, and whether it needs the parts that the
// kernels' kFull instances add: a residual, or output columns that end inside
// 16 bytes.
inline bool epilogue_full(const GemmParams &p) { return p.residual != nullptr || tma_cols(p.out_cols) != p.out_cols; }

inline int epilogue_variant(const GemmParams &p)
{
    return act_gated(p.act) ? kEpiGated : p.act != kActNone || epilogue_full(p) ? kEpiAct : kEpiPlain;
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (fn == nullptr) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }
    return fn;
}

// 2-D map over a packed FP4 operand [rows, row_bytes] with boxes of
// `box_bytes` (64 or 128) x `box_rows`, swizzled with the same width, zero
// fill outside the tensor.
inline bool make_operand_map(CUtensorMap *map, const void *base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows,
                             uint32_t box_bytes = 128)
{
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    cuuint64_t dims[2] = {row_bytes, rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {box_bytes, box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUtensorMapSwizzle swz = box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Columns of an output map: the whole 16-byte pieces (an output narrower than
// one is stored without the TMA; its map is not used).
inline uint64_t output_map_cols(int out_cols) { return out_cols >= 8 ? (uint64_t)tma_cols(out_cols) : 8; }

// Map of the bf16 output [m, n_out] (row stride ldo elements) for TMA stores
// of 16-column x 32-row boxes, no swizzle.  The TMA skips elements outside
// [0, n_out) x [0, m), columns in units of 8: n_out is a multiple of 8 (from
// output_map_cols).  Requires a 16-B aligned base and ldo % 8 == 0.
inline bool make_output_map(CUtensorMap *map, void *base, uint64_t n_out, uint64_t m, uint64_t ldo)
{
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    cuuint64_t dims[2] = {n_out, m};
    cuuint64_t strides[1] = {ldo * 2};
    cuuint32_t box[2] = {16, 32};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of the bf16 output [m, n_out] (row stride ldo elements) for TMA stores
// of 64-column x 32-row boxes (128-byte rows) with the 128-byte swizzle; the
// TMA skips elements outside [0, n_out) x [0, m), columns in units of 8.
// Requires a 16-B aligned base and ldo % 8 == 0.
inline bool make_output_map_sw128(CUtensorMap *map, void *base, uint64_t n_out, uint64_t m, uint64_t ldo)
{
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    cuuint64_t dims[2] = {n_out, m};
    cuuint64_t strides[1] = {ldo * 2};
    cuuint32_t box[2] = {64, 32};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of a tiled scale tensor viewed as [bands, band_bytes / 8] 8-byte
// elements (one row per 128-row band), for copies of `box_elems` elements of
// two consecutive bands at once (the scale tiles of one K stage of a 256-row
// operand tile); zero fill past the last band or the band's end.  band_bytes
// is a multiple of 512 and the base 16-B aligned.
inline bool make_scale_bands_map(CUtensorMap *map, const void *base, uint64_t band_bytes, uint64_t bands,
                                 uint32_t box_elems)
{
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    cuuint64_t dims[2] = {band_bytes / 8, bands};
    cuuint64_t strides[1] = {band_bytes};
    cuuint32_t box[2] = {box_elems, 2};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of a bf16 activation [m, k] (row stride ld elements) for copies of 256
// columns x 16 rows (the fused small-m linear's per-stage slice), no swizzle,
// zero fill past m and k.  Requires a 16-B aligned base and ld % 8 == 0.
inline bool make_x_slice_map(CUtensorMap *map, const void *base, uint64_t k, uint64_t m, uint64_t ld)
{
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    cuuint64_t dims[2] = {k, m};
    cuuint64_t strides[1] = {ld * 2};
    cuuint32_t box[2] = {256, 16};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D map over bf16 rows [rows, cols] (row stride ld elements) with boxes of
// 64 columns x 128 rows, 128-byte swizzle (the K-major operand layout of a
// kind::f16 MMA), zero fill outside the tensor.  Requires a 16-B aligned base
// and ld % 8 == 0.
inline bool make_bf16_rows_map(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t ld)
{
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {ld * 2};
    cuuint32_t box[2] = {64, 128};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gemm_detail
}  // namespace nvfp4
