// Rows to their experts and back, for gfx950: the gather of the tokens' rows
// in expert order, the weighted sum of the experts' outputs (combine) and its
// gradient. All are bound by bytes: each row is read and written in 16-byte
// units, a row by 8 to 256 lanes (the smallest of 8, 16, 32, 64 and 256 that
// covers it), the k rows of a token in flight together, two units of each
// where a row has that many. 8192 tokens of 8 rows of 4096 halves: 103 us
// (5.9 TB/s); a wave per token 117 to 138, without the non-temporal hint 110.
// Rows may start at any element: the units are
// plain 16-byte accesses at element alignment, which gfx950's vector memory
// takes, and a row's last partial unit goes element by element.
//
// Sums are FP32, rounded once at the store. A lane adds its terms in order and
// the lanes join in a fixed tree, so results repeat bit for bit.
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "moe.h"
#include "wide_grid.h"

namespace libgemm {
namespace {

constexpr int kRowThreads = 256;

typedef v4u unit_any __attribute__((aligned(1)));

template <typename T>
struct Unit {   // 16 bytes of T
    static constexpr int N = 16 / (int)sizeof(T);
    T e[N];
};

template <typename T>
__device__ __forceinline__ Unit<T> load_unit(const T* p) {
    return __builtin_bit_cast(Unit<T>, __builtin_nontemporal_load(reinterpret_cast<const unit_any*>(p)));
}

template <typename T>
__device__ __forceinline__ Unit<T> load_unit_cached(const T* p) {
    const v4u v = *reinterpret_cast<const unit_any*>(p);
    return __builtin_bit_cast(Unit<T>, v);
}

template <typename T>
__device__ __forceinline__ void store_unit(T* p, Unit<T> u) {
    __builtin_nontemporal_store(__builtin_bit_cast(v4u, u), reinterpret_cast<unit_any*>(p));
}

// N floats to N elements of T, in 16- or 8-byte stores.
template <typename T, int N>
__device__ __forceinline__ void store_values(T* p, const float (&v)[N]) {
    if constexpr (sizeof(T) * N == 8) {
        struct Half {
            T e[N];
        } h;
#pragma unroll
        for (int i = 0; i < N; ++i) h.e[i] = (T)v[i];
        typedef v2i any8 __attribute__((aligned(1)));
        *reinterpret_cast<any8*>(p) = __builtin_bit_cast(v2i, h);
    } else {
        constexpr int M = Unit<T>::N;
#pragma unroll
        for (int b = 0; b < N / M; ++b) {
            Unit<T> u;
#pragma unroll
            for (int i = 0; i < M; ++i) u.e[i] = (T)v[b * M + i];
            store_unit(p + b * M, u);
        }
    }
}

// The row of this lane, in a scalar register where whole waves share it.
template <int LPR>
__device__ __forceinline__ int64_t lane_row() {
    if constexpr (LPR >= kRowThreads) return wide_block();
    const int sub = threadIdx.x / LPR;
    return wide_block() * (kRowThreads / LPR) + (LPR >= 64 ? __builtin_amdgcn_readfirstlane(sub) : sub);
}

// Rows j0 .. j0 + KB - 1 of a token: each one's offset in z, -1 where there is
// none, and its weight. (No load hangs on a condition: they go out together.)
template <int KB, int LPR>
__device__ __forceinline__ void fetch_rows(const int32_t* __restrict__ row, const float* __restrict__ weight, int j0,
                                           int K, int64_t rows, int64_t width, int64_t (&at)[KB], float (&w)[KB]) {
#pragma unroll
    for (int j = 0; j < KB; ++j) {
        const int jj = min(j0 + j, K - 1);
        const int64_t r = row[jj];
        w[j] = weight ? weight[jj] : 1.0f;
        at[j] = j0 + j < K && r >= 0 && r < rows ? r * width : -1;
    }
}

// 16384 tokens of 2048 halves to 131072 rows: 141 us, 7.4 TB/s of reads and
// writes together (each token is read again for each of its 8 experts, from
// beyond the L2s). Rows picked by ranges of tokens, one range per XCD and L2,
// measured 272 us: the writes then scatter.
template <int LPR>
__global__ __launch_bounds__(kRowThreads) void moe_gather_kernel(const uint8_t* __restrict__ x,
                                                                 const int32_t* __restrict__ token,
                                                                 uint8_t* __restrict__ y, int64_t tokens,
                                                                 int64_t rows, int64_t row_bytes) {
    constexpr int U = 4;   // units in flight per lane
    const int l = threadIdx.x % LPR;
    const int64_t r = lane_row<LPR>();
    if (r >= rows) return;
    const int64_t t = token[r];
    const bool has = t >= 0 && t < tokens;
    const uint8_t* src = x + (has ? t : 0) * row_bytes;
    uint8_t* dst = y + r * row_bytes;
    const int64_t units = row_bytes / 16;
    for (int64_t u0 = l; u0 < units; u0 += LPR * U) {
        Unit<uint8_t> v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            v[i] = __builtin_bit_cast(Unit<uint8_t>, v4u{0u, 0u, 0u, 0u});
            if (has && u0 + i * LPR < units) v[i] = load_unit_cached(src + (u0 + i * LPR) * 16);
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (u0 + i * LPR < units) store_unit(dst + (u0 + i * LPR) * 16, v[i]);
    }
    for (int64_t b = units * 16 + l; b < row_bytes; b += LPR) dst[b] = has ? src[b] : (uint8_t)0;
}

// KB: rows of a token in flight (k is taken in steps of KB).
template <typename ZT, typename YT, int KB, int LPR>
__global__ __launch_bounds__(kRowThreads) void moe_combine_kernel(const ZT* __restrict__ z,
                                                                  const int32_t* __restrict__ row,
                                                                  const float* __restrict__ weight,
                                                                  YT* __restrict__ y, int64_t T, int K, int64_t rows,
                                                                  int64_t width) {
    constexpr int N = Unit<ZT>::N;
    const int l = threadIdx.x % LPR;
    const int64_t t = lane_row<LPR>();
    if (t >= T) return;
    const int32_t* rt = row + t * K;
    const float* wt = weight ? weight + t * K : nullptr;
    YT* yt = y + t * width;
    const int64_t units = width / N;
    const bool once = K <= KB;
    int64_t at[KB];
    float w[KB];
    auto fetch = [&](int j0) __attribute__((always_inline)) {
        fetch_rows<KB, LPR>(rt, wt, j0, K, rows, width, at, w);
    };
    fetch(0);
    // UN units of each row at once
    auto sum_units = [&](int64_t u, auto un) __attribute__((always_inline)) {
        constexpr int UN = decltype(un)::value;
        float acc[UN][N];
#pragma unroll
        for (int x = 0; x < UN; ++x)
#pragma unroll
            for (int i = 0; i < N; ++i) acc[x][i] = 0.0f;
        for (int j0 = 0; j0 < K; j0 += KB) {
            if (!once) fetch(j0);
            Unit<ZT> v[UN][KB];
#pragma unroll
            for (int x = 0; x < UN; ++x)
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    if (at[j] >= 0) v[x][j] = load_unit(z + at[j] + (u + x * LPR) * N);
#pragma unroll
            for (int x = 0; x < UN; ++x)
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    if (at[j] >= 0) {
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[x][i] = __builtin_fmaf(w[j], (float)v[x][j].e[i], acc[x][i]);
                    }
        }
#pragma unroll
        for (int x = 0; x < UN; ++x) store_values<YT, N>(yt + (u + x * LPR) * N, acc[x]);
    };
    int64_t u = l;
    for (; u + LPR < units; u += 2 * LPR) sum_units(u, std::integral_constant<int, 2>{});
    if (u < units) sum_units(u, std::integral_constant<int, 1>{});
    for (int64_t c = units * N + l; c < width; c += LPR) {
        float acc = 0.0f;
        for (int j0 = 0; j0 < K; j0 += KB) {
            if (!once) fetch(j0);
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (at[j] >= 0) acc = __builtin_fmaf(w[j], (float)z[at[j] + c], acc);
        }
        yt[c] = (YT)acc;
    }
}

template <typename ET, int KB, int LPR>
__global__ __launch_bounds__(kRowThreads) void moe_combine_backward_kernel(
    const ET* __restrict__ dy, const ET* __restrict__ z, const int32_t* __restrict__ row,
    const float* __restrict__ weight, ET* __restrict__ dz, float* __restrict__ dw, int64_t T, int K, int64_t rows,
    int64_t width) {
    constexpr int N = Unit<ET>::N;
    __shared__ float part[LPR > 64 ? kRowThreads / 64 * KB : 1];
    const int l = threadIdx.x % LPR;
    const int64_t t = lane_row<LPR>();
    if (t >= T) return;   // LPR > 64: the whole workgroup or none of it
    const ET* dyt = dy + t * width;
    const int64_t units = width / N;
    for (int j0 = 0; j0 < K; j0 += KB) {
        int64_t at[KB];
        float w[KB], dot[KB];
        fetch_rows<KB, LPR>(row + t * K, weight + t * K, j0, K, rows, width, at, w);
#pragma unroll
        for (int j = 0; j < KB; ++j) dot[j] = 0.0f;
        for (int64_t u = l; u < units; u += LPR) {
            const Unit<ET> d = load_unit_cached(dyt + u * N);
            Unit<ET> v[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (at[j] >= 0) v[j] = load_unit(z + at[j] + u * N);
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (at[j] >= 0) {
                    Unit<ET> o;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        dot[j] = __builtin_fmaf((float)v[j].e[i], (float)d.e[i], dot[j]);
                        o.e[i] = (ET)(w[j] * (float)d.e[i]);
                    }
                    store_unit(dz + at[j] + u * N, o);
                }
        }
        for (int64_t c = units * N + l; c < width; c += LPR) {
            const float d = (float)dyt[c];
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (at[j] >= 0) {
                    dot[j] = __builtin_fmaf((float)z[at[j] + c], d, dot[j]);
                    dz[at[j] + c] = (ET)(w[j] * d);
                }
        }
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
            for (int s = (LPR < 64 ? LPR : 64) / 2; s; s >>= 1) dot[j] += __shfl_xor(dot[j], s);
        if constexpr (LPR > 64) {
            const int wave = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int j = 0; j < KB; ++j) part[wave * KB + j] = dot[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                dot[j] = part[j];
                for (int v = 1; v < kRowThreads / 64; ++v) dot[j] += part[v * KB + j];
            }
            __syncthreads();
        }
        if (l == 0) {
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (j0 + j < K) dw[t * K + j0 + j] = at[j] >= 0 ? dot[j] : 0.0f;
        }
    }
}

// Lanes of a row of `units` units: the smallest of 8, 16, 32, 64 and 256 that
// covers it (64 up to 128 units: two each).
int lanes_for(int64_t units) {
    if (units > 128) return 256;
    for (int l = 8; l < 64; l *= 2)
        if (units <= l) return l;
    return 64;
}

dim3 blocks_for(int64_t rows, int lpr) { return wide_grid((rows + kRowThreads / lpr - 1) / (kRowThreads / lpr)); }

template <typename F>
hipError_t with_lanes(int lpr, F f) {
    switch (lpr) {
        case 8: return f(std::integral_constant<int, 8>{});
        case 16: return f(std::integral_constant<int, 16>{});
        case 32: return f(std::integral_constant<int, 32>{});
        case 64: return f(std::integral_constant<int, 64>{});
        default: return f(std::integral_constant<int, 256>{});
    }
}

template <typename F>
hipError_t with_batch(int64_t K, F f) {
    if (K <= 1) return f(std::integral_constant<int, 1>{});
    if (K <= 2) return f(std::integral_constant<int, 2>{});
    if (K <= 4) return f(std::integral_constant<int, 4>{});
    return f(std::integral_constant<int, 8>{});
}

template <typename ZT, typename YT>
hipError_t combine(const void* z, const int32_t* row, const float* weight, void* y, int64_t T, int64_t K, int64_t rows,
                   int64_t width, hipStream_t stream) {
    const int lpr = lanes_for((width + Unit<ZT>::N - 1) / Unit<ZT>::N);
    return with_batch(K, [&](auto kb) {
        return with_lanes(lpr, [&](auto lanes) {
            constexpr int L = decltype(lanes)::value;
            moe_combine_kernel<ZT, YT, decltype(kb)::value, L><<<blocks_for(T, L), kRowThreads, 0, stream>>>(
                (const ZT*)z, row, weight, (YT*)y, T, (int)K, rows, width);
            return hipGetLastError();
        });
    });
}

template <typename ET>
hipError_t combine_backward(const void* dy, const void* z, const int32_t* row, const float* weight, void* dz,
                            float* dw, int64_t T, int64_t K, int64_t rows, int64_t width, hipStream_t stream) {
    const int lpr = lanes_for((width + Unit<ET>::N - 1) / Unit<ET>::N);
    return with_batch(K, [&](auto kb) {
        return with_lanes(lpr, [&](auto lanes) {
            constexpr int L = decltype(lanes)::value;
            moe_combine_backward_kernel<ET, decltype(kb)::value, L><<<blocks_for(T, L), kRowThreads, 0, stream>>>(
                (const ET*)dy, (const ET*)z, row, weight, (ET*)dz, dw, T, (int)K, rows, width);
            return hipGetLastError();
        });
    });
}

}  // namespace

hipError_t launch_moe_gather(const void* x, const int32_t* token, void* y, int64_t tokens, int64_t rows,
                             int64_t row_bytes, hipStream_t stream) {
    if (rows == 0 || row_bytes == 0) return hipSuccess;
    return with_lanes(lanes_for((row_bytes + 15) / 16), [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        moe_gather_kernel<L><<<blocks_for(rows, L), kRowThreads, 0, stream>>>(
            (const uint8_t*)x, token, (uint8_t*)y, tokens, rows, row_bytes);
        return hipGetLastError();
    });
}

hipError_t launch_moe_combine(const void* z, int z_dtype, const int32_t* row, const float* weight, void* y,
                              int y_dtype, int64_t T, int64_t K, int64_t rows, int64_t width, hipStream_t stream) {
    if (T == 0 || width == 0) return hipSuccess;
    if (z_dtype == OUT_F16)
        return y_dtype == OUT_F16 ? combine<_Float16, _Float16>(z, row, weight, y, T, K, rows, width, stream)
                                  : combine<_Float16, float>(z, row, weight, y, T, K, rows, width, stream);
    return y_dtype == OUT_F16 ? combine<float, _Float16>(z, row, weight, y, T, K, rows, width, stream)
                              : combine<float, float>(z, row, weight, y, T, K, rows, width, stream);
}

hipError_t launch_moe_combine_backward(const void* dy, const void* z, int dtype, const int32_t* row,
                                       const float* weight, void* dz, float* dw, int64_t T, int64_t K, int64_t rows,
                                       int64_t width, hipStream_t stream) {
    if (T == 0) return hipSuccess;
    return dtype == OUT_F16 ? combine_backward<_Float16>(dy, z, row, weight, dz, dw, T, K, rows, width, stream)
                            : combine_backward<float>(dy, z, row, weight, dz, dw, T, K, rows, width, stream);
}

}  // namespace libgemm
