// Gradient to the weights of products grouped by rows, for gfx950:
//
//   C[g] = A[rows of g]^T B[rows of g]     A[rows, M], B[rows, N] FP16, C[g] M x N
//
// The sum runs over the group's rows, the slow direction of both operands, so
// both reach the matrix cores through LDS transpose reads (ds_read_b64_tr_b16),
// as row-major B does in the plain products. One workgroup computes a 128 x
// 128 tile of one group, 4 waves of 64 x 64, 64 rows at a time, registers
// ahead of two LDS stages (the layout and padding of gemm_tile_impl.h's
// row-major B). Rows past the group's end are staged as zeros on both sides
// (another group's rows may hold NaN); a group without rows gives zeros.
// Operands of any alignment are read in 16-byte pieces.
#include "gemm_tile_impl.h"

namespace libgemm {
namespace {

using WT = tile::Tile<2, 128, 128, 64, 2, 2, false>;

template <int OUT>
__global__ __launch_bounds__(256) void wgrad_tile_kernel(const _Float16* __restrict__ A,
                                                         const _Float16* __restrict__ B, void* __restrict__ C,
                                                         const int32_t* __restrict__ offsets, int groups, int rows,
                                                         int M, int N, int tiles_m, int tiles_n) {
    constexpr int BK = 64, OP = WT::B_BYTES;   // one operand's stage
    __shared__ __attribute__((aligned(16))) uint8_t smem_raw[4 * OP];
    LDS_AS uint8_t* smem = (LDS_AS uint8_t*)smem_raw;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
    int tm, tn;
    tile_coords(blockIdx.x, groups * tiles_m, tiles_n, tm, tn);
    const int grp = tm / tiles_m, m0 = (tm % tiles_m) * 128, n0 = tn * 128;
    const int lo = min(max(offsets[grp], 0), rows), hi = max(lo, min(max(offsets[grp + 1], 0), rows));
    const int nk = (hi - lo + BK - 1) / BK;

    const int srow = tid >> 4, scol = tid & 15;   // staged chunk: rows srow + 16 i, 16-byte column scol
    v4u ra[4], rb[4];
    const bool inner = m0 + 128 <= M && n0 + 128 <= N;
    auto load = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = lo + kt * BK + srow + 16 * i;
            const uint8_t* pa = reinterpret_cast<const uint8_t*>(A + (int64_t)r * M);
            const uint8_t* pb = reinterpret_cast<const uint8_t*>(B + (int64_t)r * N);
            if (inner && (kt + 1) * BK <= hi - lo) {
                ra[i] = *reinterpret_cast<const tile::v4u_any*>(pa + 2 * (m0 + 8 * scol));
                rb[i] = *reinterpret_cast<const tile::v4u_any*>(pb + 2 * (n0 + 8 * scol));
            } else {
                ra[i] = tile::load_chunk_any<2>(pa, r < hi, m0 + 8 * scol, M);
                rb[i] = tile::load_chunk_any<2>(pb, r < hi, n0 + 8 * scol, N);
            }
        }
    };
    auto store = [&](int st) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = WT::b_row(srow + 16 * i) + scol * 16;
            *(LDS_AS v4u*)(smem + 2 * st * OP + at) = ra[i];
            *(LDS_AS v4u*)(smem + (2 * st + 1) * OP + at) = rb[i];
        }
    };
    const int g = lane >> 4, j16 = lane & 15;
    const int in = WT::b_row(8 * g + (j16 >> 2)) + 8 * (j16 & 3);   // + 2 * column
    v4f acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    if (nk > 0) {
        load(0);
        store(0);
        __syncthreads();
        for (int kt = 0; kt < nk; ++kt) {
            if (kt + 1 < nk) load(kt + 1);
            const LDS_AS uint8_t* as = smem + 2 * (kt & 1) * OP + in + 2 * 64 * wm;
            const LDS_AS uint8_t* bs = smem + (2 * (kt & 1) + 1) * OP + in + 2 * 64 * wn;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                v8h bo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    bo[j] = tile::Operand<2>::read_b(bs + WT::b_row(32 * ks) + 32 * j, WT::SB);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const v8h ao = tile::Operand<2>::read_b(as + WT::b_row(32 * ks) + 32 * i, WT::SB);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ao, bo[j], acc[i][j], 0, 0, 0);
                }
            }
            if (kt + 1 < nk) store((kt + 1) & 1);
            __syncthreads();
        }
    }
    const int64_t base = (int64_t)grp * M * N;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = m0 + 64 * wm + 16 * i + 4 * g + r, col = n0 + 64 * wn + 16 * j + j16;
                if (row < M && col < N) tile::store_one<OUT>(C, base + (int64_t)row * N + col, acc[i][j][r], 0);
            }
}

}  // namespace

hipError_t launch_grouped_wgrad(const GroupedArgs& a) {
    const int64_t tiles_m = (a.M + 127) / 128, tiles_n = (a.N + 127) / 128, blocks = a.groups * tiles_m * tiles_n;
    if (blocks <= 0) return hipSuccess;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    const _Float16* A = reinterpret_cast<const _Float16*>(a.A);
    const _Float16* B = reinterpret_cast<const _Float16*>(a.B);
    if (a.out_dtype == OUT_F32)
        wgrad_tile_kernel<OUT_F32><<<(unsigned)blocks, 256, 0, a.stream>>>(
            A, B, a.C, a.offsets, (int)a.groups, (int)a.K, (int)a.M, (int)a.N, (int)tiles_m, (int)tiles_n);
    else
        wgrad_tile_kernel<OUT_F16><<<(unsigned)blocks, 256, 0, a.stream>>>(
            A, B, a.C, a.offsets, (int)a.groups, (int)a.K, (int)a.M, (int)a.N, (int)tiles_m, (int)tiles_n);
    return hipGetLastError();
}

}  // namespace libgemm
