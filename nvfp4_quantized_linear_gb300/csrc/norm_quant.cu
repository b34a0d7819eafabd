// Residual addition, RMS norm and quantization in one pass:
//   h = x + residual (fp32),  h_out = bf16(h),
//   y = (h / sqrt(mean(h^2) + eps)) * gamma  (fp32),
//   codes and scales of y in the operand format of the linear that follows.
// The norm is taken of the unrounded fp32 sum and y is not rounded to bf16 on
// its way into the codes: each value is rounded once, into its code.
//
// A CTA works on one row at a time.  A thread owns 16 consecutive elements per
// step, one NVFP4 block or half of an MX block, so block maxima, scales and
// packed codes need no shared memory; the row's fp32 values stay in registers
// between the sum of squares and the quantization, so each input byte is read
// once.
#include <cuda_bf16.h>

#include "block_launch.cuh"
#include "common.cuh"
#include "ptx.cuh"
#include "quant_core.cuh"
#include "scale_math.cuh"

namespace nvfp4 {
namespace {

using namespace quant_core;

// Scale code of an MXFP8 block (32 E4M3 elements, E8M0 scale 2^s):
// s = floor(log2 amax) - 8, the largest E4M3 exponent, clamped to +-127.
__device__ __forceinline__ uint32_t mx8_scale_code(float amax)
{
    if (amax == 0.0f) return 0;
    const int e = (int)(__float_as_uint(amax) >> 23);     // amax >= 0; a subnormal clamps to code 0 like e = 0
    return (uint32_t)max(e - 8, 0);
}

// Four fp32 to E4M3 (nearest even, saturating), the first in the lowest byte.
__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d)
{
    return cvt_e4m3x2(b, a) | (cvt_e4m3x2(d, c) << 16);
}

// fp32 of the 16 bf16 at row[k0 ..], zero past k or without a row.
__device__ __forceinline__ void load_row16(float (&v)[16], const uint16_t *row, int k0, int k, bool ok)
{
    const Raw16 r = load16(row, k0, k, ok);
    float a[8], b[8];
    unpack8(r.a, a);
    unpack8(r.b, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) { v[i] = a[i]; v[8 + i] = b[i]; }
}

// Sum over the block of one value per thread, the same in every thread and in
// a fixed order.  `part` holds 32 floats that no thread still reads.
__device__ __forceinline__ float block_sum(float v, float *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float total = 0.0f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) total += part[w];
    return total;
}

__device__ __forceinline__ float rstd_of(float sum, const NormQuantParams &p)
{
    return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(sum, (float)p.k) + p.eps));
}

__device__ __forceinline__ void zero_scale_row(const NormQuantParams &p, int row)
{
    for (int w = threadIdx.x; w < p.nbp / 4; w += blockDim.x)
        *reinterpret_cast<uint32_t *>(p.sf + sf_offset(row, 4 * w, p.nbp)) = 0;
}

// The second half of a row's work for one thread's 16 elements at k0: h, then
// y = h * rstd * gamma into codes and a scale.
template <int kFmt>
__device__ __forceinline__ void finish16(const NormQuantParams &p, int row, int k0, const float (&h)[16], float rstd,
                                         const float (&g)[16], float gs)
{
    if (p.h != nullptr && k0 < p.k) {
        uint16_t *o = p.h + (int64_t)row * p.ldh + k0;
        if (k0 + 16 <= p.k) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<uint4 *>(o + 8 * i) =
                    make_uint4(bf16x2_rn(h[8 * i], h[8 * i + 1]), bf16x2_rn(h[8 * i + 2], h[8 * i + 3]),
                               bf16x2_rn(h[8 * i + 4], h[8 * i + 5]), bf16x2_rn(h[8 * i + 6], h[8 * i + 7]));
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (k0 + i < p.k) o[i] = (uint16_t)bf16x2_rn(h[i], 0.0f);
        }
    }
    float y0[8], y1[8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y0[i] = h[i] * rstd * g[i];
        y1[i] = h[8 + i] * rstd * g[8 + i];
        amax = max_abs3(amax, y0[i], y1[i]);
    }
    uint32_t code;
    if constexpr (kFmt == kFmtNvfp4) {
        code = cvt_e4m3x2(0.0f, div6_rn(__fmul_rn(amax, gs))) & 0x7Fu;
        const float d = e4m3_to_f32(code);
        const float inv = d == 0.0f ? 0.0f : __fdiv_rn(gs, d);
        if (k0 < p.kp)
            *reinterpret_cast<uint2 *>(p.q + (int64_t)row * (p.kp / 2) + k0 / 2) =
                make_uint2(quant8(y0, inv), quant8(y1, inv));
    } else {
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));      // the block's other half
        code = kFmt == kFmtMxfp8 ? mx8_scale_code(amax) : mx_scale_code(amax);
        const float mul = mx_scale_mul(code);
        if (k0 < p.kp) {
            if constexpr (kFmt == kFmtMxfp8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) { y0[i] *= mul; y1[i] *= mul; }
                *reinterpret_cast<uint4 *>(p.q + (int64_t)row * p.kp + k0) =
                    make_uint4(cvt_e4m3x4(y0[0], y0[1], y0[2], y0[3]), cvt_e4m3x4(y0[4], y0[5], y0[6], y0[7]),
                               cvt_e4m3x4(y1[0], y1[1], y1[2], y1[3]), cvt_e4m3x4(y1[4], y1[5], y1[6], y1[7]));
            } else {
                *reinterpret_cast<uint2 *>(p.q + (int64_t)row * (p.kp / 2) + k0 / 2) =
                    make_uint2(quant8(y0, mul), quant8(y1, mul));
            }
        }
    }
    // four consecutive scale codes as one word: the blocks of 4 lanes
    // (NVFP4) or of 8 (MX, two lanes a block)
    constexpr int kStep = kFmt == kFmtNvfp4 ? 1 : 2;
    const uint32_t c1 = __shfl_down_sync(kFull, code, kStep);
    const uint32_t c2 = __shfl_down_sync(kFull, code, 2 * kStep);
    const uint32_t c3 = __shfl_down_sync(kFull, code, 3 * kStep);
    const int c = k0 / (16 * kStep);
    if (threadIdx.x % (4 * kStep) == 0 && c < p.nb)
        *reinterpret_cast<uint32_t *>(p.sf + sf_offset(row, c, p.nbp)) = code | (c1 << 8) | (c2 << 16) | (c3 << 24);
}

// One row per CTA, loaded straight into registers: few rows, or rows too long
// for the ring of the kernel below.
template <int kFmt, int U>
__global__ void __launch_bounds__(1024) norm_quant_kernel(const NormQuantParams p)
{
    __shared__ float s_part[32];
    const int tid = threadIdx.x;
    const int row = blockIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    if (row >= p.m) {                                    // padding rows of the last scale band
        zero_scale_row(p, row);
        return;
    }
    const uint16_t *x = p.x + (int64_t)row * p.ldx;
    const uint16_t *res = p.residual != nullptr ? p.residual + (int64_t)row * p.ldr : nullptr;
    float h[U][16];
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k0 = (u * blockDim.x + tid) * 16;
        load_row16(h[u], x, k0, p.k, k0 < p.k);
        if (res != nullptr) {
            float r[16];
            load_row16(r, res, k0, p.k, k0 < p.k);
#pragma unroll
            for (int i = 0; i < 16; ++i) h[u][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = __fmaf_rn(h[u][i], h[u][i], sum);
    }
    const float gs = kFmt == kFmtNvfp4 ? __ldg(p.gs) : 1.0f;
    const float rstd = rstd_of(block_sum(sum, s_part), p);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k0 = (u * blockDim.x + tid) * 16;
        float g[16];
        load_row16(g, p.gamma, k0, p.k, k0 < p.k);
        finish16<kFmt>(p, row, k0, h[u], rstd, g, gs);
    }
}

// Persistent CTAs over the rows, the next rows' x and residual arriving in a ring
// of shared memory by bulk copies while a row is worked on: without it a CTA
// loads, reduces and stores in turn, and the memory idles between the phases.
// A thread owns the same 16 columns (U steps of them) of every row and keeps
// their gamma in registers.
template <int kFmt, int U>
__global__ void __launch_bounds__(512, U == 1 ? 2 : 1) norm_quant_ring_kernel(const NormQuantParams p, int stages, uint32_t row_bytes)
{
    extern __shared__ __align__(128) uint8_t ring[];      // [stages][x row, residual row]
    __shared__ uint64_t full[kNormMaxStages];
    __shared__ float s_part[2][32];
    const int tid = threadIdx.x;
    const bool use_res = p.residual != nullptr;
    const uint32_t stage_bytes = use_res ? 2 * row_bytes : row_bytes;
    griddep_launch_dependents();
    griddep_wait();
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_mbarrier_init();
    }
    __syncthreads();
    const uint64_t pol = l2_policy_evict_first();
    auto request = [&](int row, int s) {                  // thread 0
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        bulk_load(ring + s * stage_bytes, p.x + (int64_t)row * p.ldx, row_bytes, &full[s], pol);
        if (use_res)
            bulk_load(ring + s * stage_bytes + row_bytes, p.residual + (int64_t)row * p.ldr, row_bytes, &full[s], pol);
    };
    const int step = gridDim.x;
    if (tid == 0)
        for (int s = 0; s < stages && (int)blockIdx.x + s * step < p.m; ++s) request(blockIdx.x + s * step, s);
    uint4 gamma[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Raw16 g = load16(p.gamma, (u * blockDim.x + tid) * 16, p.k, (int)(u * blockDim.x + tid) * 16 < p.k);
        gamma[u][0] = g.a;
        gamma[u][1] = g.b;
    }
    const float gs = kFmt == kFmtNvfp4 ? __ldg(p.gs) : 1.0f;
    for (int row = p.m + blockIdx.x; row < p.mp; row += step) zero_scale_row(p, row);
    int s = 0;
    uint32_t phase = 0;
    int it = 0;
    for (int row = blockIdx.x; row < p.m; row += step, ++it) {
        if (!mbar_wait(&full[s], phase, p.err_flag, kErrTimeout, kDefaultWaitNs)) {
            // expired: give the copies in flight (this row's and the next ones')
            // as long once more, then end the block
            for (int i = 0; i < stages && row + i * step < p.m; ++i)
                mbar_wait(&full[(s + i) % stages], phase ^ (s + i >= stages ? 1u : 0u), p.err_flag, kErrTimeout,
                          kDefaultWaitNs);
            return;
        }
        const uint8_t *xs = ring + s * stage_bytes;
        float h[U][16];
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k0 = (u * blockDim.x + tid) * 16;
            float v[8];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int c = k0 + 8 * half;
                if (c < p.k) {
                    unpack8(*reinterpret_cast<const uint4 *>(xs + 2 * c), v);
                    if (use_res) {
                        float r[8];
                        unpack8(*reinterpret_cast<const uint4 *>(xs + row_bytes + 2 * c), r);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] += r[i];
                    }
                    if (c + 8 > p.k)                     // the row's last piece holds bytes past k
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (c + i >= p.k) v[i] = 0.0f;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    h[u][8 * half + i] = v[i];
                    sum = __fmaf_rn(v[i], v[i], sum);
                }
            }
        }
        // after the sum's barrier every thread has read the stage: refill it
        const float rstd = rstd_of(block_sum(sum, s_part[it & 1]), p);
        if (tid == 0 && row + stages * step < p.m) request(row + stages * step, s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float g[16], a[8], b[8];
            unpack8(gamma[u][0], a);
            unpack8(gamma[u][1], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) { g[i] = a[i]; g[8 + i] = b[i]; }
            finish16<kFmt>(p, row, (u * blockDim.x + tid) * 16, h[u], rstd, g, gs);
        }
        if (++s == stages) { s = 0; phase ^= 1; }
    }
}

template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), unsigned grid, int threads, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int U>
cudaError_t launch_rows(const NormQuantParams &p, int threads, cudaStream_t s)
{
    void (*kernel)(NormQuantParams) = p.fmt == kFmtNvfp4   ? norm_quant_kernel<kFmtNvfp4, U>
                                      : p.fmt == kFmtMxfp4 ? norm_quant_kernel<kFmtMxfp4, U>
                                                           : norm_quant_kernel<kFmtMxfp8, U>;
    return launch_dependent(kernel, (unsigned)p.mp, threads, 0, s, p);
}

template <int kFmt, int U>
cudaError_t launch_ring_fmt(const NormQuantParams &p, int threads, unsigned grid, int stages, uint32_t row_bytes,
                            size_t smem, cudaStream_t s)
{
    static int configured_device = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(norm_quant_ring_kernel<kFmt, U>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNormRingBytes);
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    return launch_dependent(norm_quant_ring_kernel<kFmt, U>, grid, threads, smem, s, p, stages, row_bytes);
}

template <int U>
cudaError_t launch_ring(const NormQuantParams &p, int threads, unsigned grid, int stages, uint32_t row_bytes,
                        size_t smem, cudaStream_t s)
{
    return p.fmt == kFmtNvfp4   ? launch_ring_fmt<kFmtNvfp4, U>(p, threads, grid, stages, row_bytes, smem, s)
           : p.fmt == kFmtMxfp4 ? launch_ring_fmt<kFmtMxfp4, U>(p, threads, grid, stages, row_bytes, smem, s)
                                : launch_ring_fmt<kFmtMxfp8, U>(p, threads, grid, stages, row_bytes, smem, s);
}

}  // namespace

cudaError_t launch_norm_quant(const NormQuantParams &p, int num_sms, cudaStream_t s)
{
    // 16 elements per thread and step; the fewest steps with at most 512
    // threads, up to 1024 threads x 4 steps (k <= kNormMaxK)
    const int units = (p.k + 15) / 16;
    const int u = units <= 512 ? 1 : units <= 1024 ? 2 : 4;
    const int threads = ((units + u - 1) / u + 31) / 32 * 32;
    // The ring: CTAs of 1024 threads per SM in all (512 with two steps, whose
    // registers allow no more), each with as many rows in flight as fit, two at
    // least.
    const uint32_t row_bytes = (uint32_t)((p.k + 7) / 8 * 16);
    const uint32_t stage_bytes = p.residual != nullptr ? 2 * row_bytes : row_bytes;
    int ctas = (u == 1 ? 1024 : 512) / threads;
    if (ctas > 16) ctas = 16;
    if (ctas < 1) ctas = 1;
    while (ctas > 1 && kNormRingBytes / ctas / stage_bytes < 2) --ctas;
    int stages = (int)(kNormRingBytes / ctas / stage_bytes);
    if (stages > kNormMaxStages) stages = kNormMaxStages;
    if (u <= 2 && stages >= 2 && p.m > ctas * num_sms) {
        const size_t smem = (size_t)stages * stage_bytes;
        const unsigned grid = (unsigned)(ctas * num_sms);
        return u == 1 ? launch_ring<1>(p, threads, grid, stages, row_bytes, smem, s)
                      : launch_ring<2>(p, threads, grid, stages, row_bytes, smem, s);
    }
    return u == 1 ? launch_rows<1>(p, threads, s) : u == 2 ? launch_rows<2>(p, threads, s) : launch_rows<4>(p, threads, s);
}

}  // namespace nvfp4
