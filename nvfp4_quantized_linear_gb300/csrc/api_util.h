// Host-side argument checks shared by the C-ABI translation units.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "nvfp4.h"

namespace nvfp4 {
namespace api {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;

// Records a printf-style reason as this thread's last error and returns `st`.
nvfp4_status fail(nvfp4_status st, const char *fmt, ...);
// Clears the last error and returns NVFP4_OK.
nvfp4_status ok();
// NVFP4_OK and the SM count if the current device can run the kernels.
nvfp4_status current_device(int *num_sms);
// A launch's result as a status ("<what> launch failed: ...").
nvfp4_status launch_status(cudaError_t e, const char *what);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The bytes [lo, hi) an argument covers.
struct Range {
    uintptr_t lo, hi;
    const char *name;
};

inline Range range(const void *p, size_t bytes, const char *name)
{
    uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + bytes, name};
}

// Strided 2-D bf16 matrix: rows x cols elements, row stride ld elements.
inline Range range2d(const void *p, int64_t rows, int64_t cols, int64_t ld, const char *name)
{
    size_t bytes = p != nullptr && rows > 0 ? (size_t)((rows - 1) * ld + cols) * 2 : 0;
    return range(p, bytes, name);
}

// NVFP4_ERR_ALIAS if an output overlaps an input or another output.
nvfp4_status check_aliases(const Range *outs, int n_out, const Range *ins, int n_in);

// A bf16 matrix argument: non-null, row stride at least `cols`, rows on 16-byte
// boundaries.
nvfp4_status check_rows(const void *p, int64_t cols, int64_t ld, const char *name);

}  // namespace api
}  // namespace nvfp4
