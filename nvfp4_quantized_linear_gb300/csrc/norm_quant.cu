// Residual addition, RMS norm and quantization in one pass:
//   h = x + residual (fp32),  h_out = bf16(h),
//   y = (h / sqrt(mean(h^2) + eps)) * gamma  (fp32),
//   codes and scales of y in the operand format of the linear that follows.
// The norm is taken of the unrounded fp32 sum and y is not rounded to bf16 on
// its way into the codes: each value is rounded once, into its code.
//
// One CTA per row.  A thread owns 16 consecutive elements per step, one NVFP4
// block or half of an MX block, so block maxima, scales and packed codes need
// no shared memory; the row's fp32 values stay in registers between the sum of
// squares and the quantization, so each input byte is read once.
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

template <int kFmt, int U>
__global__ void __launch_bounds__(1024) norm_quant_kernel(const NormQuantParams p)
{
    __shared__ float s_part[32];
    const int tid = threadIdx.x;
    const int row = blockIdx.x;
    if (row >= p.m) {                                    // padding rows of the last scale band
        for (int w = tid; w < p.nbp / 4; w += blockDim.x)
            *reinterpret_cast<uint32_t *>(p.sf + sf_offset(row, 4 * w, p.nbp)) = 0;
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
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if ((tid & 31) == 0) s_part[tid >> 5] = sum;
    __syncthreads();
    float total = 0.0f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) total += s_part[w];
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(total, (float)p.k) + p.eps));

    const float gs = kFmt == kFmtNvfp4 ? __ldg(p.gs) : 1.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k0 = (u * blockDim.x + tid) * 16;
        if (p.h != nullptr && k0 < p.k) {
            uint16_t *o = p.h + (int64_t)row * p.ldh + k0;
            if (k0 + 16 <= p.k) {
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    *reinterpret_cast<uint4 *>(o + 8 * g) =
                        make_uint4(bf16x2_rn(h[u][8 * g], h[u][8 * g + 1]), bf16x2_rn(h[u][8 * g + 2], h[u][8 * g + 3]),
                                   bf16x2_rn(h[u][8 * g + 4], h[u][8 * g + 5]),
                                   bf16x2_rn(h[u][8 * g + 6], h[u][8 * g + 7]));
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (k0 + i < p.k) o[i] = (uint16_t)bf16x2_rn(h[u][i], 0.0f);
            }
        }
        float g[16];
        load_row16(g, p.gamma, k0, p.k, k0 < p.k);
        float y0[8], y1[8];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y0[i] = h[u][i] * rstd * g[i];
            y1[i] = h[u][8 + i] * rstd * g[8 + i];
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
        if (tid % (4 * kStep) == 0 && c < p.nb)
            *reinterpret_cast<uint32_t *>(p.sf + sf_offset(row, c, p.nbp)) = code | (c1 << 8) | (c2 << 16) | (c3 << 24);
    }
}

template <int U>
cudaError_t launch_fmt(const NormQuantParams &p, int threads, cudaStream_t s)
{
    void (*kernel)(NormQuantParams) = p.fmt == kFmtNvfp4   ? norm_quant_kernel<kFmtNvfp4, U>
                                      : p.fmt == kFmtMxfp4 ? norm_quant_kernel<kFmtMxfp4, U>
                                                           : norm_quant_kernel<kFmtMxfp8, U>;
    kernel<<<(unsigned)p.mp, threads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_quant(const NormQuantParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    // 16 elements per thread and step; the fewest steps with at most 512
    // threads, up to 1024 threads x 4 steps (k <= kNormMaxK)
    const int units = (p.k + 15) / 16;
    const int u = units <= 512 ? 1 : units <= 1024 ? 2 : 4;
    const int threads = ((units + u - 1) / u + 31) / 32 * 32;
    return u == 1 ? launch_fmt<1>(p, threads, s) : u == 2 ? launch_fmt<2>(p, threads, s) : launch_fmt<4>(p, threads, s);
}

}  // namespace nvfp4
