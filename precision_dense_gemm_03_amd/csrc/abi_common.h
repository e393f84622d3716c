// Argument checks shared by the C-ABI translation units (host only).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "libgemm.h"

namespace libgemm {

constexpr int64_t kMaxDim = 0x7FFFFFFF;

inline bool dim_ok(int64_t d) { return d >= 0 && d <= kMaxDim; }

// Byte counts are formed only after this check: an operand of 2^62 bytes or
// more is a GEMM_ERR_DIM (no device holds one), so every later product of a
// dimension pair and an element size fits in int64.
constexpr unsigned __int128 kMaxBytes = (unsigned __int128)1 << 62;
inline bool bytes_ok(int64_t a, int64_t b, int64_t es) {
    if (a < 0 || b < 0) return false;
    return (unsigned __int128)a * (unsigned __int128)b * (unsigned __int128)es < kMaxBytes;
}

// Byte ranges [p, p+n) and [q, q+m) overlap (empty ranges never do).
inline bool overlaps(const void* p, int64_t n, const void* q, int64_t m) {
    if (!p || !q || n <= 0 || m <= 0) return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

inline int64_t out_size(int out_dtype) {
    return out_dtype == GEMM_OUT_F32 ? 4 : (out_dtype == GEMM_OUT_F16 ? 2 : 1);
}

inline bool fp8_out(int out_dtype) { return out_dtype == GEMM_OUT_E4M3 || out_dtype == GEMM_OUT_E5M2; }

// GEMM_OK when the current device is gfx950 (looked up once per device).
int check_device();

inline int status_of(hipError_t e) {
    if (e == hipSuccess) return GEMM_OK;
    (void)hipGetLastError();
    return GEMM_ERR_LAUNCH;
}

}  // namespace libgemm
