// 8-bit values with a power-of-two scale per 32 (row_io.h): from FP32 or FP16, and
// back. One pass, bound by bytes: a lane takes 8 values, four lanes a block. 8192 x
// 4096 FP16: 18.5 us, 5.5 TB/s (16.4 with the input in the Infinity Cache, back 16.8);
// 4099 columns 21.
#include "kernels.h"
#include "norm.h"
#include "row_io.h"
#include "wide_grid.h"

namespace libgemm {

namespace {

constexpr int kThreads = 256;

// Eight values as they lie in memory (n of them exist, the others are zeros).
template <int T>
__device__ __forceinline__ void load_raw(const void* base, int64_t at, int n, uint32_t (&w)[T == OUT_F16 ? 4 : 8]) {
    constexpr int W = T == OUT_F16 ? 4 : 8;
    if (n >= 8) {
#pragma unroll
        for (int k = 0; k < W / 4; ++k) {
            const v4u v = T == OUT_F16 ? *reinterpret_cast<const v4u_b1*>(reinterpret_cast<const _Float16*>(base) + at)
                                       : *reinterpret_cast<const v4u_b1*>(reinterpret_cast<const float*>(base) + at + 4 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * k + i] = v[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= n) continue;
        if constexpr (T == OUT_F16)
            w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(base)[at + i] << (16 * (i & 1));
        else
            w[i] = reinterpret_cast<const uint32_t*>(base)[at + i];
    }
}

// The four lanes that hold a block of 32 agree on its exponent, and each gives its 8
// codes. FP16 magnitudes are compared as 16-bit integers, two at a time; a block with
// an infinity, a NaN or a value above the format's bound is looked at again.
template <int T, int FMT>
__device__ __forceinline__ int block_codes(uint32_t (&w)[T == OUT_F16 ? 4 : 8], uint32_t& lo, uint32_t& hi) {
    if constexpr (T == OUT_F16) {
        typedef uint16_t v2u16 __attribute__((ext_vector_type(2)));
        constexpr uint32_t top = FMT == FMT_E5M2 ? 0x7B00u : 0x7B80u;   // 57344, 61440
        auto largest = [&]() __attribute__((always_inline)) -> uint32_t {
            v2u16 m = {0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(v2u16, w[i] & 0x7FFF7FFFu));
            return max((uint32_t)m[0], (uint32_t)m[1]);
        };
        uint32_t m = largest();
        const uint32_t before[4] = {w[0], w[1], w[2], w[3]};
        if (__builtin_amdgcn_ballot_w64(m > top) != 0) {
            m = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int sh = 16 * (i & 1);
                const uint32_t x = before[i / 2] >> sh & 0xFFFFu, a = x & 0x7FFFu;
                const uint32_t y = a > top && a < 0x7C00u ? (x & 0x8000u) | top : x;
                w[i / 2] = (w[i / 2] & ~(0xFFFFu << sh)) | (y << sh);
                if (a < 0x7C00u) m = max(m, y & 0x7FFFu);
            }
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
        const int e = mx_exponent<FMT>((float)__builtin_bit_cast(_Float16, (uint16_t)m));
        const float power = mx_power(e);
        lo = mx_pack4_f16<FMT>(w[0], w[1], power);
        hi = mx_pack4_f16<FMT>(w[2], w[3], power);
        return e;
    } else {
        float v[8], m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = bits_f32(w[i]);
            m = fmaxf(m, finite_abs(v[i]));
        }
        m = fmaxf(m, __shfl_xor(m, 1, 64));
        m = fmaxf(m, __shfl_xor(m, 2, 64));
        const int e = mx_exponent<FMT>(m);
        const float power = mx_power(e);
        lo = mx_pack4<FMT>(v[0], v[1], v[2], v[3], power);
        hi = mx_pack4<FMT>(v[4], v[5], v[6], v[7], power);
        return e;
    }
}

// Whole blocks in a row (cols % 32 == 0): x and q are one run of blocks, U units of
// 8 values in flight per lane.
template <int T, int FMT, int U>
__global__ __launch_bounds__(kThreads) void mx_flat_kernel(const void* __restrict__ x, int64_t units,
                                                           uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
    const int64_t first = wide_block() * (kThreads * U) + threadIdx.x;
    uint32_t w[U][T == OUT_F16 ? 4 : 8];
#pragma unroll
    for (int u = 0; u < U; ++u)   // (past the end: the last unit again)
        load_raw<T>(x, min(first + u * kThreads, units - 1) * 8, 8, w[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t at = first + u * kThreads;
        uint32_t lo, hi;
        const int e = block_codes<T, FMT>(w[u], lo, hi);
        if (at >= units) continue;
        *reinterpret_cast<v2u_b1*>(q + at * 8) = v2u{lo, hi};
        if ((threadIdx.x & 3) == 0) scale[at >> 2] = (uint8_t)(e + 127);
    }
}

// Any width: a wave goes along a row, 512 values at a time (its strip's, where rows
// are few: row_grid).
template <int T, int FMT>
__global__ __launch_bounds__(kThreads) void mx_rows_kernel(const void* __restrict__ x, int64_t rows, int64_t cols,
                                                           uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
    const int lane = threadIdx.x & 63;
    const int64_t blocks = (cols + kMxBlock - 1) / kMxBlock, step = (int64_t)gridDim.x * (kThreads / 64);
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); r < rows; r += step)
        for (int64_t c0 = 512 * (int64_t)blockIdx.y; c0 < cols; c0 += 512 * (int64_t)gridDim.y) {
            const int64_t c = c0 + 8 * lane, left = cols - c;
            const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
            uint32_t w[T == OUT_F16 ? 4 : 8], lo, hi;
            load_raw<T>(x, r * cols + c, n, w);
            const int e = block_codes<T, FMT>(w, lo, hi);
            if (n > 0) {
                store_codes8(q + r * cols + c, n, lo, hi);
                if ((lane & 3) == 0) scale[r * blocks + c / kMxBlock] = (uint8_t)(e + 127);
            }
        }
}

template <int FMT, int T>
__global__ __launch_bounds__(kThreads) void mx_unpack_kernel(const uint8_t* __restrict__ q,
                                                             const uint8_t* __restrict__ scale, int64_t rows,
                                                             int64_t cols, void* __restrict__ y) {
    const int lane = threadIdx.x & 63;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 64);
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); r < rows; r += step)
        for (int64_t c = 512 * (int64_t)blockIdx.y + 8 * lane; c < cols; c += 512 * (int64_t)gridDim.y) {
            float v[8];
            load_row8<FMT == FMT_E5M2 ? OUT_E5M2 : OUT_E4M3>(q, scale, r, c, cols, v);
            store8<T>(y, r * cols + c, cols - c >= 8 ? 8 : (int)(cols - c), v);
        }
}

// Workgroups of four rows each, as many as keep the chip busy; few rows are cut into
// strips of 512 columns and more.
dim3 row_grid(int64_t rows, int64_t cols) {
    const int64_t most = 256 * 16, n = (rows + 3) / 4, strips = (cols + 511) / 512;
    if (n >= most) return dim3((unsigned)most);
    const int64_t room = most / n;
    return dim3((unsigned)n, (unsigned)(strips < room ? strips : room));
}

template <int T, int FMT>
hipError_t pack(const void* x, int64_t rows, int64_t cols, uint8_t* q, uint8_t* scale, hipStream_t s) {
    constexpr int U = T == OUT_F16 ? 4 : 2;
    if (cols % kMxBlock == 0) {
        const int64_t units = rows * (cols / 8);
        // A lane alone with its loads where there are few.
        const bool few = units < (int64_t)256 * kThreads * 4 * U;
        const int64_t per = kThreads * (few ? 1 : U), blocks = (units + per - 1) / per;
        if (few) mx_flat_kernel<T, FMT, 1><<<wide_grid(blocks), kThreads, 0, s>>>(x, units, q, scale);
        else mx_flat_kernel<T, FMT, U><<<wide_grid(blocks), kThreads, 0, s>>>(x, units, q, scale);
    } else {
        mx_rows_kernel<T, FMT><<<row_grid(rows, cols), kThreads, 0, s>>>(x, rows, cols, q, scale);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_mx(const void* x, int dtype, int64_t rows, int64_t cols, int fmt, uint8_t* q,
                              uint8_t* scale, hipStream_t s) {
    if (dtype == OUT_F16)
        return fmt == FMT_E5M2 ? pack<OUT_F16, FMT_E5M2>(x, rows, cols, q, scale, s)
                               : pack<OUT_F16, FMT_E4M3>(x, rows, cols, q, scale, s);
    return fmt == FMT_E5M2 ? pack<OUT_F32, FMT_E5M2>(x, rows, cols, q, scale, s)
                           : pack<OUT_F32, FMT_E4M3>(x, rows, cols, q, scale, s);
}

hipError_t launch_dequantize_mx(const uint8_t* q, const uint8_t* scale, int fmt, int64_t rows, int64_t cols, void* y,
                                int dtype, hipStream_t s) {
    const dim3 grid = row_grid(rows, cols);
#define LIBGEMM_GO(FMT, T) mx_unpack_kernel<FMT, T><<<grid, kThreads, 0, s>>>(q, scale, rows, cols, y)
    if (fmt == FMT_E5M2) {
        if (dtype == OUT_F16) LIBGEMM_GO(FMT_E5M2, OUT_F16);
        else LIBGEMM_GO(FMT_E5M2, OUT_F32);
    } else {
        if (dtype == OUT_F16) LIBGEMM_GO(FMT_E4M3, OUT_F16);
        else LIBGEMM_GO(FMT_E4M3, OUT_F32);
    }
#undef LIBGEMM_GO
    return hipGetLastError();
}

}  // namespace libgemm
