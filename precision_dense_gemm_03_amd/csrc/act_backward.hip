// Gradient of a product's epilogue y = act(z) + residual, z = product + bias:
//
//   dz = dy act'(z),   dbias[j] = sum over rows of dz[., j]
//
// z as FP32, FP16 or 8-bit values (row_io.h), which are widened as they are loaded.
// One pass over dy and z, bound by bytes. A workgroup takes a strip of up to 512
// columns (8 per lane) and every gridDim.y-th set of rows, kRows rows of a lane in
// flight; the column sums stay in registers (FP32, of dz before it is rounded), the
// waves' sums meet in LDS, and each workgroup leaves one row of partial sums that a
// second launch adds in a fixed order.
//
// 8192 x 12288 FP16 from E4M3 z, GELU: 102 to 106 us with the column sums, 5.0 TB/s
// (FP16 z 120, 5.0 TB/s); without an activation 79. 1001 x 1416: 6 + 3.4 us, latency.
#include "act.h"
#include "kernels.h"
#include "norm.h"
#include "row_io.h"

namespace libgemm {

namespace {

constexpr int kRows = 4;
constexpr int64_t kWantBlocks = 256 * 8;

// Lanes that share a row of a strip.
int lanes_of(int64_t cols) {
    int n = 1;
    while (n < 64 && 8 * n < cols) n *= 2;
    return n;
}

// MODE: rows of whole pieces of eight, rows that cut the last one (Piece8), rows of
// fewer than eight columns.
enum { WHOLE = 0, CUT = 1, NARROW = 2 };

template <int T, int Z, int ACT, int MODE>
__global__ __launch_bounds__(256) void act_backward_kernel(ActBackwardArgs a, int lpr) {
    __shared__ float sums[256][8];
    const int tid = threadIdx.x, sub = tid / lpr, subs = 256 / lpr;   // rows side by side in the workgroup
    const int64_t first = (int64_t)blockIdx.x * lpr * 8;              // of the strip's columns
    const Piece8 p(first + tid % lpr * 8, MODE == NARROW ? 8 : a.cols);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    const int64_t step = (int64_t)gridDim.y * subs * kRows;
    int64_t r0 = (int64_t)blockIdx.y * subs * kRows + sub;
    if constexpr (MODE == NARROW) {
        const int n = (int)a.cols;
        for (; r0 < a.rows; r0 += step)
            for (int u = 0; u < kRows; ++u) {
                const int64_t r = r0 + u * subs;
                if (r >= a.rows) break;
                float d[8], x[8];
                load8<T>(a.dy, r * n, n, 1.0f, d);
                if constexpr (ACT != ACT_NONE) load_row8<Z>(a.z, a.zscale, r, 0, n, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (ACT != ACT_NONE) d[i] *= slope<ACT>(x[i]);
                    acc[i] += d[i];
                }
                if (a.dz) store8<T>(a.dz, r * n, n, d);
            }
    } else if (p.skip < 8) {
        // every load first; rows past the end are the last one and count for nothing
        for (; r0 < a.rows; r0 += step) {
            Raw8<T> dy[kRows];
            Raw8<Z> z[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int64_t r = min(r0 + u * subs, a.rows - 1);
                fetch8<T, MODE == CUT>(dy[u], a.dy, nullptr, r, a.cols, p);
                if constexpr (ACT != ACT_NONE) fetch8<Z, MODE == CUT>(z[u], a.z, a.zscale, r, a.cols, p);
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                if (r0 + u * subs >= a.rows) break;
                float d[8], x[8];
                values8<T, MODE == CUT>(dy[u], p.skip, d);
                if constexpr (ACT != ACT_NONE) values8<Z, MODE == CUT>(z[u], p.skip, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (ACT != ACT_NONE) d[i] *= slope<ACT>(x[i]);
                    acc[i] += d[i];
                }
                if (a.dz) store8<T>(a.dz, (r0 + u * subs) * a.cols + p.at, 8, d);
            }
        }
    }
    if (!a.partial) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[tid][i] = acc[i];
    __syncthreads();
    for (int j = tid; j < 8 * lpr; j += 256) {
        const int64_t col = first + j;
        if (col >= a.cols) break;
        // (a cut piece's own columns are its last)
        const int64_t past = first + j / 8 * 8 + 8 - a.cols;
        const int e = j % 8 + (MODE == CUT && past > 0 ? (int)past : 0);
        float s = 0.0f;
        for (int g = 0; g < subs; ++g) s += sums[g * lpr + j / 8][e];
        a.partial[(int64_t)blockIdx.y * a.cols + col] = s;
    }
}

// 32 columns per workgroup (8 lanes of four), the parts over 32 lanes each.
__global__ __launch_bounds__(256) void sum_parts_kernel(const float* __restrict__ partial, int64_t parts, int64_t cols,
                                                        int64_t first, float* __restrict__ out) {
    __shared__ float sums[32][33];
    const int l = threadIdx.x & 7, g = threadIdx.x >> 3;
    const int64_t c = first + (int64_t)blockIdx.x * 32 + 4 * l;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c + 4 <= cols) {
#pragma unroll 8
        for (int64_t p = g; p < parts; p += 32) {
            const v4u v = *reinterpret_cast<const v4u_b1*>(partial + p * cols + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += bits_f32(v[i]);
        }
    } else {
        for (int64_t p = g; p < parts; p += 32)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < cols) s[i] += partial[p * cols + c + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[g][4 * l + i] = s[i];
    __syncthreads();
    if (threadIdx.x < 32) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += sums[i][threadIdx.x];
        const int64_t col = first + (int64_t)blockIdx.x * 32 + threadIdx.x;
        if (col < cols) out[col] = t;
    }
}

template <int T, int Z>
hipError_t act_backward(const ActBackwardArgs& a, int act, float* dbias, hipStream_t s) {
    const int lpr = lanes_of(a.cols);
    const int64_t strips = (a.cols + 8 * lpr - 1) / (8 * lpr), parts = act_backward_parts(a.rows, a.cols);
    const dim3 grid((unsigned)strips, (unsigned)parts);
#define LIBGEMM_GO(ACT)                                                                            \
    do {                                                                                           \
        if (a.cols < 8) act_backward_kernel<T, Z, ACT, NARROW><<<grid, 256, 0, s>>>(a, lpr);       \
        else if (a.cols % 8) act_backward_kernel<T, Z, ACT, CUT><<<grid, 256, 0, s>>>(a, lpr);     \
        else act_backward_kernel<T, Z, ACT, WHOLE><<<grid, 256, 0, s>>>(a, lpr);                   \
    } while (0)
    switch (act) {
        case ACT_RELU: LIBGEMM_GO(ACT_RELU); break;
        case ACT_GELU: LIBGEMM_GO(ACT_GELU); break;
        case ACT_GELU_TANH: LIBGEMM_GO(ACT_GELU_TANH); break;
        case ACT_SILU: LIBGEMM_GO(ACT_SILU); break;
        default: LIBGEMM_GO(ACT_NONE); break;
    }
#undef LIBGEMM_GO
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.partial) e = launch_sum_parts(a.partial, parts, a.cols, dbias, s);
    return e;
}

}  // namespace

hipError_t launch_sum_parts(const float* partial, int64_t parts, int64_t cols, float* out, hipStream_t s) {
    const int64_t blocks = (cols + 31) / 32;
    for (int64_t at = 0; at < blocks; at += 1 << 22) {
        const int64_t n = blocks - at < (1 << 22) ? blocks - at : (1 << 22);
        sum_parts_kernel<<<(unsigned)n, 256, 0, s>>>(partial, parts, cols, at * 32, out);
    }
    return hipGetLastError();
}

int64_t act_backward_parts(int64_t rows, int64_t cols) {
    const int lpr = lanes_of(cols);
    const int64_t strips = (cols + 8 * lpr - 1) / (8 * lpr), sets = 256 / lpr * kRows;
    const int64_t all = (rows + sets - 1) / sets, want = (kWantBlocks + strips - 1) / strips;
    const int64_t n = all < want ? all : want;
    return n < 1 ? 1 : (n < 1024 ? n : 1024);
}

hipError_t launch_act_backward(const ActBackwardArgs& a, int dtype, int z_dtype, int act, float* dbias, hipStream_t s) {
    if (a.rows <= 0 || a.cols <= 0) return hipSuccess;
#define LIBGEMM_GO(T)                                                            \
    switch (z_dtype) {                                                           \
        case OUT_F32: return act_backward<T, OUT_F32>(a, act, dbias, s);         \
        case OUT_F16: return act_backward<T, OUT_F16>(a, act, dbias, s);         \
        case OUT_E4M3: return act_backward<T, OUT_E4M3>(a, act, dbias, s);       \
        default: return act_backward<T, OUT_E5M2>(a, act, dbias, s);             \
    }
    if (dtype == OUT_F16) {
        LIBGEMM_GO(OUT_F16)
    }
    LIBGEMM_GO(OUT_F32)
#undef LIBGEMM_GO
}

}  // namespace libgemm
