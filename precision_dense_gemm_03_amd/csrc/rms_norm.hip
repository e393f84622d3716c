// Root-mean-square norm with the residual's addition, and its gradient:
//
//   h = round(x + residual), rstd = 1 / sqrt(mean(h^2) + eps), y = h w rstd
//   n = h rstd, g = w dy:  dx = rstd (g - n mean(g n)) + dh,  dw[j] = sum over rows of dy n
//
// y as FP32 or FP16, or as FP8 codes with one scale per row for the products that
// scale rows: scale = max|y| / fmax (or the power of two), code = FP8(y / scale)
// formed as (h w) (rstd / scale), one FP32 factor. max|y| is max|h w| rstd, so the
// sum of squares and the maximum take one reduction, and a row one trip through
// registers: each byte is read and written once, and bytes bound the kernels.
//
// A row belongs to 1, 4 or 8 waves (W), which hold CH chunks of 8 values per lane;
// workgroups go over rows with the weights in registers, so the gradient to the
// weights is summed in registers too, and each workgroup leaves one row of partial
// sums, added by a second launch in a fixed order (no atomics: results repeat).
// Rows of more than 16384 values are read twice, the second time from beyond the L2
// again: 2048 x 32768 FP16 with a residual into E4M3 127 us for 102 at 4096 x 16384 (516
// MiB read where the operands are 256), its gradient joined by dh 177 for 112 (two
// launches, 258 and 386 MiB).
//
// 16384 x 4096 FP16 with a residual into E4M3: 89 us, 5.3 TB/s (a copy of 1 GiB 5.2 to
// 5.4); 16 rows 3.9 us, latency. Gradient, 8192 x 4096 FP16 joined by dh: 55 us with
// the sums over rows (52 + 4), 5.1 TB/s.
#include "kernels.h"
#include "norm.h"
#include "row_io.h"
#include "wide_grid.h"

namespace libgemm {

namespace {

constexpr int64_t kMostWidth = 8 * 64 * 8 * 4;   // values of a row that registers hold (8 waves, 4 chunks)

template <int OUT>
constexpr bool is_fp8 = OUT == OUT_E4M3 || OUT == OUT_E5M2;

// Sum (a) and maximum (b) over the W waves of a row; red: W pairs per row of the
// workgroup, used in turn by two halves so that one barrier is enough.
template <int W>
__device__ __forceinline__ void row_reduce(float& a, float& b, float (*red)[2], int wave) {
    a = wave_sum(a);
    b = wave_max(b);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) {
            red[wave][0] = a;
            red[wave][1] = b;
        }
        __syncthreads();
        a = red[0][0];
        b = red[0][1];
#pragma unroll
        for (int i = 1; i < W; ++i) {
            a += red[i][0];
            b = max_nan(b, red[i][1]);
        }
    }
}

template <int W>
__device__ __forceinline__ float row_sum(float a, float* red, int wave) {
    a = wave_sum(a);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) red[wave] = a;
        __syncthreads();
        a = red[0];
#pragma unroll
        for (int i = 1; i < W; ++i) a += red[i];
    }
    return a;
}

// x + residual rounded to the stream's type.
template <int T>
__device__ __forceinline__ void add8(float (&v)[8], const float (&r)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = T == OUT_F16 ? (float)(_Float16)(v[i] + r[i]) : v[i] + r[i];
}

// The row's scale and the factor that takes h w to what is stored. lift: h w is so
// small that the factor would pass FP32's range; it is then for h w 2^100 (the
// quotient is below 2^125 even with the least scale).
constexpr float kLift = 0x1p100f;
template <int OUT>
__device__ __forceinline__ float row_factor(float rstd, float most, int pow2, float& scale, bool& lift) {
    lift = false;
    if constexpr (!is_fp8<OUT>) return rstd;
    scale = scale_for_format(most * rstd, OUT == OUT_E5M2 ? FMT_E5M2 : FMT_E4M3, pow2);
    const float factor = rstd / scale;
    lift = factor == __builtin_inff() && rstd < __builtin_inff();
    return lift ? rstd * (1.0f / kLift) / scale : factor;
}

template <int OUT>
__device__ __forceinline__ void store_y(void* y, int64_t at, int n, const float (&v)[8], float factor) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i] * factor;
    if constexpr (is_fp8<OUT>) {
        constexpr int F = OUT == OUT_E5M2 ? FMT_E5M2 : FMT_E4M3;
        store_codes8(reinterpret_cast<uint8_t*>(y) + at, n, fp8_pack4<F>(o[0], o[1], o[2], o[3]),
                     fp8_pack4<F>(o[4], o[5], o[6], o[7]));
    } else {
        store8<OUT>(y, at, n, o);
    }
}

__device__ __forceinline__ int count8(int64_t c, int64_t width) {
    const int64_t left = width - c;
    return left >= 8 ? 8 : (left > 0 ? (int)left : 0);
}

// MODE: rows of whole pieces of eight columns, rows that cut the last one (Piece8),
// rows of fewer than eight.
enum { WHOLE = 0, CUT = 1, NARROW = 2 };

// A row's pieces in a lane's registers: piece k at column first + 512 W k. They are
// loaded without conditions (one past the row's end is its last) and all before the
// first is looked at; what is no piece is zeros.
template <int T, int W, int CH, int MODE>
struct Chunks {
    Raw8<T> raw[MODE == NARROW ? 1 : CH];
    float v[CH][8];

    __device__ __forceinline__ void fetch(const void* base, const uint8_t* scales, int64_t r, int64_t width, int first) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = first + k * 512 * W;
            if constexpr (MODE == NARROW) load_row8<T>(base, scales, r, c, width, v[k]);
            else fetch8<T, MODE == CUT>(raw[k], base, scales, r, width, Piece8(c, width));
        }
    }

    __device__ __forceinline__ void values(int64_t width, int first) {
        if constexpr (MODE != NARROW) {
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const Piece8 p(first + k * 512 * W, width);
                values8<T, MODE == CUT>(raw[k], p.skip, v[k]);
                if (p.skip >= 8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[k][i] = 0.0f;
                }
            }
        }
    }
};

// Where a lane's piece k is stored and how many values of it; and whether value i
// counts in a row's sums (a cut piece's first values are another lane's).
template <int W, int MODE>
struct Place {
    int64_t at;
    int n, skip;
    __device__ __forceinline__ Place(int first, int k, int64_t width) {
        const int c = first + k * 512 * W;
        if constexpr (MODE == NARROW) {
            at = c;
            n = c < width ? (int)width : 0;
            skip = 0;
        } else {
            const Piece8 p(c, width);
            at = p.at;
            skip = p.skip;
            n = skip < 8 ? 8 : 0;
        }
    }
    __device__ __forceinline__ bool counts(int i) const { return MODE != CUT || i >= skip; }
};

// W waves per row (W = 1: four rows per workgroup), CH chunks per lane. Lane l of
// the row's W * 64 takes chunks l, l + 64 W, ..
template <int T, int OUT, int W, int CH, int MODE>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void rms_norm_kernel(NormArgs a) {
    constexpr int RPW = W == 1 ? 4 : 1;
    __shared__ float red[2][W][2];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int first = 8 * (W == 1 ? lane : (int)threadIdx.x);
    Chunks<OUT_F32, W, CH, MODE> weight;
    weight.fetch(a.weight, nullptr, 0, a.width, first);
    weight.values(a.width, first);
    float (&w)[CH][8] = weight.v;
    int half = 0;
    for (int64_t r = (int64_t)blockIdx.x * RPW + (W == 1 ? wave : 0); r < a.rows; r += (int64_t)gridDim.x * RPW) {
        const int64_t base = r * a.width;
        Chunks<T, W, CH, MODE> x, res;
        x.fetch(a.x, nullptr, r, a.width, first);
        if (a.residual) res.fetch(a.residual, nullptr, r, a.width, first);
        x.values(a.width, first);
        float (&v)[CH][8] = x.v;
        if (a.residual) {
            res.values(a.width, first);
#pragma unroll
            for (int k = 0; k < CH; ++k) add8<T>(v[k], res.v[k]);
        }
        float sum = 0.0f, most = 0.0f;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const Place<W, MODE> p(first, k, a.width);
            if (a.h && p.n) store8<T>(a.h, base + p.at, MODE == NARROW ? p.n : 8, v[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (p.counts(i)) sum = __builtin_fmaf(v[k][i], v[k][i], sum);
                v[k][i] *= w[k][i];
                if constexpr (is_fp8<OUT>) most = max_nan(most, __builtin_fabsf(v[k][i]));
            }
        }
        if constexpr (is_fp8<OUT>) row_reduce<W>(sum, most, red[half], wave);
        else sum = row_sum<W>(sum, &red[half][0][0], wave);
        half ^= 1;
        const float rstd = 1.0f / __builtin_sqrtf(sum * a.inv_width + a.eps);
        float scale = 1.0f;
        bool lift;
        const float factor = row_factor<OUT>(rstd, most, a.pow2, scale, lift);
        if (is_fp8<OUT> && lift) {
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] *= kLift;
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const Place<W, MODE> p(first, k, a.width);
            if (p.n) store_y<OUT>(a.y, base + p.at, MODE == NARROW ? p.n : 8, v[k], factor);
        }
        if (first == 0) {
            if (a.rstd) a.rstd[r] = rstd;
            if constexpr (is_fp8<OUT>) a.scale[r] = scale;
        }
    }
}

// Rows that registers do not hold: read twice.
template <int T, int OUT>
__global__ __launch_bounds__(512) void rms_norm_long_kernel(NormArgs a) {
    __shared__ float red[2][8][2];
    const int wave = threadIdx.x >> 6;
    int half = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t base = r * a.width;
        auto value = [&](int64_t c, int n, float (&v)[8]) {
            load8<T>(a.x, base + c, n, 1.0f, v);
            if (a.residual) {
                float s[8];
                load8<T>(a.residual, base + c, n, 1.0f, s);
                add8<T>(v, s);
            }
        };
        float sum = 0.0f, most = 0.0f;
        for (int64_t c = 8 * threadIdx.x; c < a.width; c += 8 * 512) {
            const int n = count8(c, a.width);
            float v[8], w[8], part = 0.0f;
            value(c, n, v);
            load8<OUT_F32>(a.weight, c, n, 1.0f, w);
            if (a.h) store8<T>(a.h, base + c, n, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                part = __builtin_fmaf(v[i], v[i], part);
                most = max_nan(most, __builtin_fabsf(v[i] * w[i]));
            }
            sum += part;
        }
        row_reduce<8>(sum, most, red[half], wave);
        half ^= 1;
        const float rstd = 1.0f / __builtin_sqrtf(sum * a.inv_width + a.eps);
        float scale = 1.0f;
        bool lift;
        const float factor = row_factor<OUT>(rstd, most, a.pow2, scale, lift);
        for (int64_t c = 8 * threadIdx.x; c < a.width; c += 8 * 512) {
            const int n = count8(c, a.width);
            float v[8], w[8];
            value(c, n, v);
            load8<OUT_F32>(a.weight, c, n, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= lift ? w[i] * kLift : w[i];
            store_y<OUT>(a.y, base + c, n, v, factor);
        }
        if (threadIdx.x == 0) {
            if (a.rstd) a.rstd[r] = rstd;
            if constexpr (is_fp8<OUT>) a.scale[r] = scale;
        }
    }
}

// ---------------------------------------------------------------- gradient

// T: type of dy, dh and dx; H: of h (8-bit values with scales among them).
template <int T, int H, int W, int CH, int MODE>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void rms_norm_backward_kernel(NormBackwardArgs a) {
    constexpr int RPW = W == 1 ? 4 : 1;
    __shared__ float red[2][W];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int first = 8 * (W == 1 ? lane : (int)threadIdx.x);
    Chunks<OUT_F32, W, CH, MODE> weight;
    weight.fetch(a.weight, nullptr, 0, a.width, first);
    weight.values(a.width, first);
    float (&w)[CH][8] = weight.v;
    float dw[CH][8];   // (of a cut piece's first values both lanes have the whole sum)
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
    int half = 0;
    for (int64_t r = (int64_t)blockIdx.x * RPW + (W == 1 ? wave : 0); r < a.rows; r += (int64_t)gridDim.x * RPW) {
        const int64_t base = r * a.width;
        Chunks<H, W, CH, MODE> hh;
        Chunks<T, W, CH, MODE> gg, dd;
        const float rstd = a.rstd[r];
        hh.fetch(a.h, a.hscale, r, a.width, first);
        gg.fetch(a.dy, nullptr, r, a.width, first);
        if (a.dh) dd.fetch(a.dh, nullptr, r, a.width, first);
        hh.values(a.width, first);
        gg.values(a.width, first);
        float (&n)[CH][8] = hh.v;
        float (&g)[CH][8] = gg.v;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const Place<W, MODE> p(first, k, a.width);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[k][i] *= rstd;
                dw[k][i] = __builtin_fmaf(g[k][i], n[k][i], dw[k][i]);
                g[k][i] *= w[k][i];
                if (p.counts(i)) sum = __builtin_fmaf(g[k][i], n[k][i], sum);
            }
        }
        const float mean = row_sum<W>(sum, red[half], wave) * a.inv_width;
        half ^= 1;
        if (a.dh) dd.values(a.width, first);
        float (&d)[CH][8] = dd.v;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const Place<W, MODE> p(first, k, a.width);
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = rstd * __builtin_fmaf(-n[k][i], mean, g[k][i]);
                if (a.dh) o[i] += d[k][i];
            }
            if (p.n) store8<T>(a.dx, base + p.at, MODE == NARROW ? p.n : 8, o);
        }
    }
    if (!a.partial) return;
    if constexpr (W == 1) {   // the workgroup's four rows meet, in order
        __shared__ float rest[3][CH][8][64];
        if (wave > 0) {
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) rest[wave - 1][k][i][lane] = dw[k][i];
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[k][i] += rest[q][k][i][lane];
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const Place<W, MODE> p(first, k, a.width);
        if (p.n) store8<OUT_F32>(a.partial, (int64_t)blockIdx.x * a.width + p.at, MODE == NARROW ? p.n : 8, dw[k]);
    }
}

// Long rows: mean(g n) of each row into the first `rows` words of the workspace,
// then dx and the weights' partial sums, a workgroup for 2048 columns and every
// gridDim.y-th row.
template <int T, int H>
__global__ __launch_bounds__(512) void rms_norm_backward_dot_kernel(NormBackwardArgs a, float* __restrict__ dots) {
    __shared__ float red[2][8];
    const int wave = threadIdx.x >> 6;
    int half = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float rstd = a.rstd[r];
        float sum = 0.0f;
        for (int64_t c = 8 * threadIdx.x; c < a.width; c += 8 * 512) {
            const int cnt = count8(c, a.width);
            float n[8], g[8], w[8], part = 0.0f;
            load_row8<H>(a.h, a.hscale, r, c, a.width, n);
            load8<T>(a.dy, r * a.width + c, cnt, 1.0f, g);
            load8<OUT_F32>(a.weight, c, cnt, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) part = __builtin_fmaf(g[i] * w[i], n[i] * rstd, part);
            sum += part;
        }
        sum = row_sum<8>(sum, red[half], wave);
        half ^= 1;
        if (threadIdx.x == 0) dots[r] = sum * a.inv_width;
    }
}

template <int T, int H>
__global__ __launch_bounds__(256) void rms_norm_backward_long_kernel(NormBackwardArgs a, const float* __restrict__ dots) {
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= a.width) return;
    const int cnt = count8(c, a.width);
    float w[8], dw[8];
    load8<OUT_F32>(a.weight, c, cnt, 1.0f, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0.0f;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float rstd = a.rstd[r], mean = dots[r];
        float n[8], g[8], o[8];
        load_row8<H>(a.h, a.hscale, r, c, a.width, n);
        load8<T>(a.dy, r * a.width + c, cnt, 1.0f, g);
        if (a.dh) load8<T>(a.dh, r * a.width + c, cnt, 1.0f, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            n[i] *= rstd;
            dw[i] = __builtin_fmaf(g[i], n[i], dw[i]);
            const float d = rstd * __builtin_fmaf(-n[i], mean, g[i] * w[i]);
            o[i] = a.dh ? d + o[i] : d;
        }
        store8<T>(a.dx, r * a.width + c, cnt, o);
    }
    if (a.partial) store8<OUT_F32>(a.partial, (int64_t)blockIdx.y * a.width + c, cnt, dw);
}

// Waves of a row and chunks of a lane that hold a row of this width, f(W, CH).
template <class F>
void by_width(int64_t width, F f) {
    if (width <= 512) f(IntC<1>{}, IntC<1>{});
    else if (width <= 1024) f(IntC<1>{}, IntC<2>{});
    else if (width <= 2048) f(IntC<4>{}, IntC<1>{});
    else if (width <= 4096) f(IntC<4>{}, IntC<2>{});
    else if (width <= 6144) f(IntC<4>{}, IntC<3>{});
    else if (width <= 8192) f(IntC<8>{}, IntC<2>{});
    else if (width <= 12288) f(IntC<8>{}, IntC<3>{});
    else f(IntC<8>{}, IntC<4>{});   // (16 waves and 2 chunks: the gradient 158 us for 118 at 4096 x 16384)
}

template <int T, int OUT>
hipError_t norm_forward(const NormArgs& a, hipStream_t s) {
    const int64_t most = 256 * 16;
    if (a.width > kMostWidth) {
        rms_norm_long_kernel<T, OUT><<<(unsigned)(a.rows < most ? a.rows : most), 512, 0, s>>>(a);
        return hipGetLastError();
    }
    by_width(a.width, [&](auto w, auto ch) {
        constexpr int W = decltype(w)::value, CH = decltype(ch)::value, RPW = W == 1 ? 4 : 1;
        const int64_t blocks = (a.rows + RPW - 1) / RPW;
        const unsigned grid = (unsigned)(blocks < most ? blocks : most), nt = W == 1 ? 256 : 64 * W;
        if (a.width % 8 == 0) {
            rms_norm_kernel<T, OUT, W, CH, WHOLE><<<grid, nt, 0, s>>>(a);
        } else if (a.width > 8) {
            rms_norm_kernel<T, OUT, W, CH, CUT><<<grid, nt, 0, s>>>(a);
        } else {
            if constexpr (W * CH == 1) rms_norm_kernel<T, OUT, W, CH, NARROW><<<grid, nt, 0, s>>>(a);
        }
    });
    return hipGetLastError();
}

template <int T, int H>
hipError_t norm_backward(const NormBackwardArgs& a, float* dweight, hipStream_t s) {
    int64_t parts = 0;
    NormBackwardArgs b = a;
    if (a.width > kMostWidth) {
        float* dots = b.partial;   // (the workspace holds the rows' words first)
        b.partial = dweight ? dots + a.rows : nullptr;
        rms_norm_backward_dot_kernel<T, H><<<(unsigned)(a.rows < 4096 ? a.rows : 4096), 512, 0, s>>>(b, dots);
        const int64_t strips = (a.width + 2047) / 2048;
        parts = norm_backward_parts(a.rows, a.width);
        rms_norm_backward_long_kernel<T, H><<<dim3((unsigned)strips, (unsigned)parts), 256, 0, s>>>(b, dots);
    } else {
        if (!dweight) b.partial = nullptr;
        by_width(a.width, [&](auto w, auto ch) {
            constexpr int W = decltype(w)::value, CH = decltype(ch)::value;
            parts = norm_backward_parts(a.rows, a.width);
            constexpr unsigned nt = W == 1 ? 256 : 64 * W;
            if (a.width % 8 == 0) {
                rms_norm_backward_kernel<T, H, W, CH, WHOLE><<<(unsigned)parts, nt, 0, s>>>(b);
            } else if (a.width > 8) {
                rms_norm_backward_kernel<T, H, W, CH, CUT><<<(unsigned)parts, nt, 0, s>>>(b);
            } else {
                if constexpr (W * CH == 1) rms_norm_backward_kernel<T, H, W, CH, NARROW><<<(unsigned)parts, nt, 0, s>>>(b);
            }
        });
    }
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && dweight) e = launch_sum_parts(b.partial, parts, a.width, dweight, s);
    return e;
}

}  // namespace

int64_t norm_backward_parts(int64_t rows, int64_t width) {
    if (width > kMostWidth) {
        const int64_t strips = (width + 2047) / 2048, want = (2048 + strips - 1) / strips;
        return rows < want ? rows : want;
    }
    const int64_t sets = width <= 1024 ? (rows + 3) / 4 : rows;   // (four rows per workgroup)
    // Each part is a row of sums written and read again. 16384 x 4096, FP16 / 8-bit h: 101
    // / 70 us with 512, 111 / 81 with 1024, 117 / 111 with 256; 4096 x 16384: 118 / 121
    // with 256, 129 / 131 with 512.
    const int64_t most = width <= 8192 ? 512 : 256;
    return sets < most ? sets : most;
}

int64_t norm_backward_words(int64_t rows, int64_t width, bool dweight) {
    return (dweight ? norm_backward_parts(rows, width) * width : 0) + (width > kMostWidth ? rows : 0);
}

hipError_t launch_rms_norm(const NormArgs& a, int dtype, int out_dtype, hipStream_t s) {
    if (a.rows <= 0 || a.width <= 0) return hipSuccess;
#define LIBGEMM_GO(T)                                                             \
    switch (out_dtype) {                                                          \
        case OUT_F32: return norm_forward<T, OUT_F32>(a, s);                      \
        case OUT_F16: return norm_forward<T, OUT_F16>(a, s);                      \
        case OUT_E4M3: return norm_forward<T, OUT_E4M3>(a, s);                    \
        default: return norm_forward<T, OUT_E5M2>(a, s);                          \
    }
    if (dtype == OUT_F16) {
        LIBGEMM_GO(OUT_F16)
    }
    LIBGEMM_GO(OUT_F32)
#undef LIBGEMM_GO
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, int dtype, int h_dtype, float* dweight, hipStream_t s) {
#define LIBGEMM_GO(T)                                                             \
    switch (h_dtype) {                                                            \
        case OUT_F32: return norm_backward<T, OUT_F32>(a, dweight, s);            \
        case OUT_F16: return norm_backward<T, OUT_F16>(a, dweight, s);            \
        case OUT_E4M3: return norm_backward<T, OUT_E4M3>(a, dweight, s);          \
        default: return norm_backward<T, OUT_E5M2>(a, dweight, s);                \
    }
    if (dtype == OUT_F16) {
        LIBGEMM_GO(OUT_F16)
    }
    LIBGEMM_GO(OUT_F32)
#undef LIBGEMM_GO
}

}  // namespace libgemm
