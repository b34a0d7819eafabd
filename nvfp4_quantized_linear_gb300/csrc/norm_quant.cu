// Residual addition, RMS norm and quantization in one pass:
//   h = x + residual (fp32),  h_out = bf16(h),
//   y = (h / sqrt(mean(h^2) + eps)) * gamma  (fp32),
//   codes and scales of y in the operand format of the linear that follows.
// The norm is taken of the unrounded fp32 sum and y is not rounded to bf16 on
// its way into the codes: each value is rounded once, into its code.
//
// A CTA works on one row at a time.  A thread owns 16 consecutive elements per
// step, one NVFP4 block or half of an MX block, so block maxima, scales and
// packed codes need no shared memory; the row's fp32 values stay with their thread
// between the sum of squares and the quantization, so each input byte is read
// once.  They stay in registers up to k = 16384 (64 registers for two steps of 16, 16
// bytes of MXFP8's spilled); the instances of four steps, for longer rows, hold 1024
// threads at 64 registers and spill 224 bytes a thread.
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

// A thread's 16 values as eight fp32 pairs (packed arithmetic, epilogue.cuh).
using Pairs = uint64_t[8];

__device__ __forceinline__ void pairs_of(Pairs &v, const Raw16 &r)
{
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf16x2_to_f32x2(w[i]);
}

// h (+)= residual, and its sum of squares.
__device__ __forceinline__ void add_pairs(Pairs &h, const Raw16 &r)
{
    Pairs v;
    pairs_of(v, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = add2(h[i], v[i]);
}

__device__ __forceinline__ float sum_squares(const Pairs &h, float sum)
{
    uint64_t s = pack2(sum, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma2(h[i], h[i], s);
    float lo, hi;
    unpack2(s, lo, hi);
    return lo + hi;
}

// Sum over the block (kWarps warps at most) of one value per thread, the same in
// every thread and in a fixed order.  `part` holds kWarps floats that no thread
// still reads, zeros past the block's warps.  Every thread adds the warps' sums
// itself: one shared-memory latency where a second round of shuffles takes five.
template <int kWarps>
__device__ __forceinline__ float block_sum(float v, float *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    uint64_t a = 0, b = 0;                               // (two floats each)
#pragma unroll
    for (int i = 0; i < kWarps / 4; ++i) {
        const ulonglong2 w = reinterpret_cast<const ulonglong2 *>(part)[i];
        a = add2(a, w.x);
        b = add2(b, w.y);
    }
    float s0, s1;
    unpack2(add2(a, b), s0, s1);
    return s0 + s1;
}

// 1 / sqrt(sum / k + eps): the approximate root r of the rounded mean + eps, and
// one Newton step whose residual 1 - a r^2 has the remainders of the product with
// 1 / k, of the sum with eps and of the square in it, so that only the last
// addition rounds.  A row's codes share this error: the IEEE quotient and root
// instead, each rounded by itself, put 81 codes of 4096 x 4096 on the wrong side of
// a threshold (an exact form's codes taken as right), this 42, and it is shorter:
// 16384 x 5120 without a residual takes 47.4 us instead of 49.7.
__device__ __forceinline__ float rstd_of(float sum, const NormQuantParams &p)
{
    const float mean = __fmul_rn(sum, p.inv_k);
    const float mean_lo = __fmaf_rn(sum, p.inv_k, -mean) + sum * p.inv_k_lo;
    const float a = __fadd_rn(mean, p.eps);
    const float added = __fsub_rn(a, mean);              // what the sum took of eps, and of the mean
    const float a_lo = __fadd_rn(__fsub_rn(mean, __fsub_rn(a, added)), __fsub_rn(p.eps, added)) + mean_lo;
    const float r = rsqrtf(a);
    const float rr = __fmul_rn(r, r);
    const float e = __fmaf_rn(-a, rr, 1.0f) - a * __fmaf_rn(r, r, -rr) - a_lo * rr;
    return fabsf(e) < 1.0f ? __fmaf_rn(0.5f * r, e, r) : r;   // (an infinite or zero mean has no residual)
}

__device__ __forceinline__ void zero_scale_row(const NormQuantParams &p, int row)
{
    for (int w = threadIdx.x; w < p.nbp / 4; w += blockDim.x)
        *reinterpret_cast<uint32_t *>(p.sf + sf_offset(row, 4 * w, p.nbp)) = 0;
}

// The second half of a row's work for one thread's 16 elements at k0: h, then
// y = (h * gamma) * rstd into codes and a scale.
template <int kFmt>
__device__ __forceinline__ void finish16(const NormQuantParams &p, int row, int k0, const Pairs &h, float rstd,
                                         const Raw16 &gamma, float gs)
{
    if (p.h != nullptr && k0 < p.k) {
        uint16_t *o = p.h + (int64_t)row * p.ldh + k0;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = bf16x2_of(h[i]);
        if (k0 + 16 <= p.k && (reinterpret_cast<uintptr_t>(o) & 31) == 0) {
            st_global_v8(o, w);                           // two 16-byte stores would each fill half of 32 sectors
        } else if (k0 + 16 <= p.k) {
            *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4 *>(o + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (k0 + i < p.k) o[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
    Pairs y;
    pairs_of(y, gamma);
    const uint64_t rs = pack2(rstd, rstd);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = mul2(mul2(h[i], y[i]), rs);                // h gamma is exact in most cases: 8 bits by few more
        float lo, hi;
        unpack2(y[i], lo, hi);
        amax = max_abs3(amax, lo, hi);
    }
    uint32_t code;
    float mul;                                            // y * mul is rounded to the element format
    if constexpr (kFmt == kFmtNvfp4) {
        code = cvt_e4m3x2(0.0f, div6_rn(__fmul_rn(amax, gs))) & 0x7Fu;
        const float d = e4m3_to_f32(code);
        mul = d == 0.0f ? 0.0f : __fdiv_rn(gs, d);
    } else {
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));      // the block's other half
        code = kFmt == kFmtMxfp8 ? mx8_scale_code(amax) : mx_scale_code(amax);
        mul = mx_scale_mul(code);
    }
    if (k0 < p.kp) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) unpack2(mul2(y[i], pack2(mul, mul)), v[2 * i], v[2 * i + 1]);
        if constexpr (kFmt == kFmtMxfp8) {
            *reinterpret_cast<uint4 *>(p.q + (int64_t)row * p.kp + k0) =
                make_uint4(cvt_e4m3x4(v[0], v[1], v[2], v[3]), cvt_e4m3x4(v[4], v[5], v[6], v[7]),
                           cvt_e4m3x4(v[8], v[9], v[10], v[11]), cvt_e4m3x4(v[12], v[13], v[14], v[15]));
        } else {
            *reinterpret_cast<uint2 *>(p.q + (int64_t)row * (p.kp / 2) + k0 / 2) =
                make_uint2(cvt_e2m1x8(*reinterpret_cast<float(*)[8]>(v)), cvt_e2m1x8(*reinterpret_cast<float(*)[8]>(v + 8)));
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
    __shared__ __align__(16) float s_part[32];
    const int tid = threadIdx.x;
    const int row = blockIdx.x;
    if (tid < 32 && tid >= blockDim.x / 32) s_part[tid] = 0.0f;
    griddep_launch_dependents();
    griddep_wait();
    if (row >= p.m) {                                    // padding rows of the last scale band
        for (int r = row; r < p.mp; r += gridDim.x - p.m) zero_scale_row(p, r);
        return;
    }
    const uint16_t *x = p.x + (int64_t)row * p.ldx;
    const uint16_t *res = p.residual != nullptr ? p.residual + (int64_t)row * p.ldr : nullptr;
    Pairs h[U];
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k0 = (u * blockDim.x + tid) * 16;
        pairs_of(h[u], load16_coherent(x, k0, p.k));
        if (res != nullptr) add_pairs(h[u], load16_coherent(res, k0, p.k));
        sum = sum_squares(h[u], sum);
    }
    const float gs = kFmt == kFmtNvfp4 ? *p.gs : 1.0f;
    Raw16 gamma = load16_coherent(p.gamma, tid * 16, p.k);       // the first step's, before the sum's barrier
    const float rstd = rstd_of(block_sum<32>(sum, s_part), p);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k0 = (u * blockDim.x + tid) * 16;
        if (u > 0) gamma = load16_coherent(p.gamma, k0, p.k);
        finish16<kFmt>(p, row, k0, h[u], rstd, gamma, gs);
    }
}

// The 16 bf16 of a copied row at k0; a row's last 16-byte piece holds bytes past k.
__device__ __forceinline__ Raw16 ring16(const uint8_t *row, int k0, int k)
{
    Raw16 r;
    r.a = r.b = make_uint4(0, 0, 0, 0);
    if (k0 + 16 <= k) {
        r.a = *reinterpret_cast<const uint4 *>(row + 2 * k0);
        r.b = *reinterpret_cast<const uint4 *>(row + 2 * k0 + 16);
    } else if (k0 < k) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t v = k0 + 2 * i < k ? *reinterpret_cast<const uint32_t *>(row + 2 * k0 + 4 * i) : 0u;
            w[i] = k0 + 2 * i + 1 < k ? v : v & 0xFFFFu;
        }
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
        r.b = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return r;
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
    __shared__ __align__(16) float s_part[2][16];
    const int tid = threadIdx.x;
    if (tid < 32 && tid % 16 >= blockDim.x / 32) s_part[tid / 16][tid % 16] = 0.0f;
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
    auto request = [&](uint32_t row, int s) {             // thread 0
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        bulk_load(ring + s * stage_bytes, p.x + (int64_t)row * p.ldx, row_bytes, &full[s], pol);
        if (use_res)
            bulk_load(ring + s * stage_bytes + row_bytes, p.residual + (int64_t)row * p.ldr, row_bytes, &full[s], pol);
    };
    // (row numbers with the steps past the last one go beyond 2^31: unsigned)
    const uint32_t step = gridDim.x, m = (uint32_t)p.m;
    if (tid == 0)
        for (int s = 0; s < stages && blockIdx.x + s * step < m; ++s) request(blockIdx.x + s * step, s);
    Raw16 gamma[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k0 = (u * blockDim.x + tid) * 16;
        gamma[u] = load16_coherent(p.gamma, k0, p.k);
    }
    const float gs = kFmt == kFmtNvfp4 ? *p.gs : 1.0f;
    for (uint32_t row = m + blockIdx.x; row < (uint32_t)p.mp; row += step) zero_scale_row(p, (int)row);
    int s = 0;
    uint32_t phase = 0;
    int it = 0;
    for (uint32_t row = blockIdx.x; row < m; row += step, ++it) {
        if (!mbar_wait(&full[s], phase, p.err_flag, kErrTimeout, kDefaultWaitNs)) {
            // expired: give the copies in flight (this row's and the next ones')
            // as long once more, then end the block
            for (int i = 0; i < stages && row + i * step < m; ++i)
                mbar_wait(&full[(s + i) % stages], phase ^ (s + i >= stages ? 1u : 0u), p.err_flag, kErrTimeout,
                          kDefaultWaitNs);
            return;
        }
        const uint8_t *xs = ring + s * stage_bytes;
        Pairs h[U];
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k0 = (u * blockDim.x + tid) * 16;
            pairs_of(h[u], ring16(xs, k0, p.k));
            if (use_res) add_pairs(h[u], ring16(xs + row_bytes, k0, p.k));
            sum = sum_squares(h[u], sum);
        }
        // after the sum's barrier every thread has read the stage: refill it
        const float rstd = rstd_of(block_sum<16>(sum, s_part[it & 1]), p);
        if (tid == 0 && row + stages * step < m) request(row + stages * step, s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            finish16<kFmt>(p, (int)row, (u * blockDim.x + tid) * 16, h[u], rstd, gamma[u], gs);
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
    // a block per row and up to 16 for the padding rows: a dependent GEMM starts
    // on the SMs that no block occupies
    return launch_dependent(kernel, (unsigned)(p.m + std::min(16, p.mp - p.m)), threads, 0, s, p);
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
    int ctas = std::max(1, std::min(32, (u == 1 ? 1024 : 512) / threads));
    auto fitting = [&](int n) { return (int)((kNormRingBytes - n * kNormCtaBytes) / n / stage_bytes); };
    while (ctas > 1 && fitting(ctas) < 2) --ctas;
    const int stages = std::min(fitting(ctas), kNormMaxStages);
    if (u <= 2 && stages >= 2 && p.m > ctas * num_sms) {
        NormQuantParams q = p;
        const cudaError_t e = device_error_word(&q.err_flag);
        if (e != cudaSuccess) return e;
        const size_t smem = (size_t)stages * stage_bytes;
        const unsigned grid = (unsigned)(ctas * num_sms);
        return u == 1 ? launch_ring<1>(q, threads, grid, stages, row_bytes, smem, s)
                      : launch_ring<2>(q, threads, grid, stages, row_bytes, smem, s);
    }
    return u == 1 ? launch_rows<1>(p, threads, s) : u == 2 ? launch_rows<2>(p, threads, s) : launch_rows<4>(p, threads, s);
}

}  // namespace nvfp4
