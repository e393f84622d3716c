// Argument checks shared by the C-ABI translation units (host only).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>

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

struct Range {
    const void* p;
    int64_t n;
};

// Every written range against every other range.
template <int W, int R>
bool aliased(const Range (&written)[W], const Range (&read)[R]) {
    for (int i = 0; i < W; ++i) {
        for (int j = 0; j < R; ++j)
            if (overlaps(written[i].p, written[i].n, read[j].p, read[j].n)) return true;
        for (int j = i + 1; j < W; ++j)
            if (overlaps(written[i].p, written[i].n, written[j].p, written[j].n)) return true;
    }
    return false;
}

constexpr int64_t kMaxRowGroups = 4096;

// The product kernels count rows, columns and K in 32 bits up to the end of a
// tile (which starts at any row of a group) or of the steps loaded ahead: less
// than 2^16 past the size.
inline bool size_ok(int64_t d) { return d >= 0 && d <= ((int64_t)1 << 31) - (1 << 16); }

inline bool fmt_ok(int f) { return f == GEMM_FMT_E4M3 || f == GEMM_FMT_E5M2; }

// a * b * c * es below the byte limit, with a * b below 2^62 first.
inline bool bytes3_ok(int64_t a, int64_t b, int64_t c, int64_t es) { return bytes_ok(a, b, es) && bytes_ok(a * b, c, es); }

// The answer of the host-only queries.
inline int put_name(const char* name, char* buf, int buflen) {
    if (!buf || buflen <= 0) return GEMM_ERR_NULL;
    std::snprintf(buf, (size_t)buflen, "%s", name);
    return GEMM_OK;
}

}  // namespace libgemm
