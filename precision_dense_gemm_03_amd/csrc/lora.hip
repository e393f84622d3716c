// The low-rank values of per-row adapters, for gfx950:
//
//   low[i, r] = lscale[a_i] sum_k X[i, k] LA[a_i, r, k]      (FP32)
//
// zero for rows without an adapter and for r from rank to rank_p (the next
// multiple of 8); the product kernels add low LB^T (lora_extra.h).
//
// Three kernels:
//
// Few rows (lora_low_dot_kernel): each usually has its own adapter, so nothing
// is shared between rows and a wave takes one (i, r): a dot product over K, both
// sides read in 16-byte pieces, rows * rank waves.
//
// More rows, 16-byte aligned (lora_low_ring_kernel): 16 rows against 16, 32 or
// 64 of an adapter's rows on the deep-ring kernel, whose direct loads take whole
// lines of both and run far ahead: the call is bound by moving X and, for each
// 16 rows again, LA into the compute units (4096 rows, K 4096, rank 64: 640 KB
// each; blocks of 64 rows, which move 256 KB, measured the same). A block's
// adapters are shared out over kLowParts workgroups, one pass each; an
// adapter's pass stores its own rows. Where the blocks leave compute units
// idle, K is cut into slices, each with its own array of sums, which every
// tile of the product adds up (4096 x 4096 x 4096, rank 64, two slices: 155.4 us
// for both launches, one 156.3).
//
// Any alignment (lora_low_kernel): a workgroup takes 16 rows and its 8 waves
// share out K in tiles of 64, straight from memory to the matrix cores; every
// adapter present multiplies the block (LA as the first operand, so a lane ends
// with one row's four neighbouring values) and its rows keep the result; the
// waves' sums join in LDS in wave order. Its loads take a line per lane: 41 us
// for the sizes above.
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "gemm_ring_impl.h"
#include "kernels.h"
#include "wide_grid.h"

namespace libgemm {
namespace {

typedef v4u any16 __attribute__((aligned(2)));

// Eight halves from k on, zero from K on.
__device__ __forceinline__ v8h chunk8(const _Float16* row, int k, int K) {
    if (k + 8 <= K) return __builtin_bit_cast(v8h, *reinterpret_cast<const any16*>(row + k));
    v8h v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? row[k + i] : (_Float16)0.0f;
    return v;
}

__global__ __launch_bounds__(256) void lora_low_dot_kernel(const _Float16* __restrict__ X,
                                                           const _Float16* __restrict__ LA,
                                                           const int32_t* __restrict__ adapter,
                                                           const float* __restrict__ lscale, int64_t waves, int K,
                                                           int rank, int rank_p, int adapters,
                                                           float* __restrict__ low) {
    const int lane = threadIdx.x & 63;
    const int64_t w = wide_block() * 4 + (threadIdx.x >> 6);
    if (w >= waves) return;
    const int64_t row = w / rank_p;
    const int r = (int)(w % rank_p);
    const int a = adapter[row];
    const bool has = a >= 0 && a < adapters && r < rank;
    float sum = 0.0f;
    if (has) {
        const _Float16* x = X + row * K;
        const _Float16* l = LA + ((int64_t)a * rank + r) * K;
        constexpr int U = 8;   // pairs of loads in flight
        for (int k0 = 8 * lane; k0 < K; k0 += 512 * U) {
            v8h xv[U], lv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + 512 * u;
                xv[u] = lv[u] = v8h{0, 0, 0, 0, 0, 0, 0, 0};
                if (k < K) {
                    xv[u] = chunk8(x, k, K);
                    lv[u] = chunk8(l, k, K);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = __builtin_fmaf((float)xv[u][i], (float)lv[u][i], sum);
        }
#pragma unroll
        for (int s = 32; s; s >>= 1) sum += __shfl_xor(sum, s);
    }
    if (lane == 0) low[row * rank_p + r] = has ? sum * lscale[a] : 0.0f;
}

// Stores the low-rank values of the rows whose adapter is `a`.
struct LowStore {
    static constexpr bool kActive = false, kStores = true;
    float* low;
    const int32_t* adapter;
    float scale;
    int a, rank, rank_p;
    __device__ __forceinline__ void store4(v4f y, int row, int col) const {
        if (col >= rank_p || adapter[row] != a) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = col + e < rank ? y[e] * scale : 0.0f;
        *reinterpret_cast<v4f*>(low + (int64_t)row * rank_p + col) = y;
    }
};

constexpr int kLowParts = 4, kLowDotRows = 64;

template <int BN>
__global__ __launch_bounds__(256) void lora_low_ring_kernel(const uint8_t* __restrict__ X,
                                                            const uint8_t* __restrict__ LA,
                                                            const int32_t* __restrict__ adapter,
                                                            const float* __restrict__ lscale, int M, int K, int rank,
                                                            int rank_p, int adapters, int parts, int kslice,
                                                            float* __restrict__ low) {
    // K tiles per barrier and stages (LDS for two workgroups per compute unit)
    constexpr int BM = 16, P = BN == 64 ? 2 : 4, S = BN == 64 ? 6 : 12;
    using T = ring::Ring<2, BM, BN, true, S>;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[T::S * T::STAGE];
    __shared__ v4f red[T::RED_SLOTS];
    const int lane = threadIdx.x & 63, m0 = blockIdx.x * BM, n0 = blockIdx.y * BN;
    const int z = blockIdx.z / parts, mypart = blockIdx.z - z * parts, k0 = z * kslice;
    low += (int64_t)z * M * rank_p;
    int mine = -1;
    if (lane < BM && m0 + lane < M) {
        mine = adapter[m0 + lane];
        if (mine < 0 || mine >= adapters) mine = -1;
    }
    if (mypart == 0) {   // rows without an adapter: zeros
        const uint64_t none = __builtin_amdgcn_ballot_w64(mine < 0);
        for (int i = threadIdx.x; i < BM * BN; i += 256) {
            const int r = i / BN, c = n0 + i % BN;
            if (((none >> r) & 1) && m0 + r < M && c < rank_p) low[(int64_t)(m0 + r) * rank_p + c] = 0.0f;
        }
    }
    int part = 0;
    for (uint64_t left = __builtin_amdgcn_ballot_w64(mine >= 0); left; part = part + 1 == parts ? 0 : part + 1) {
        const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
        left &= ~__builtin_amdgcn_ballot_w64(mine == a);
        if (part != mypart) continue;
        const LowStore store{low, adapter, lscale[a], a, rank, rank_p};
        ring::ring_body<2, BM, BN, OUT_F32, 0, 0, true, S, true, LowStore, P>(
            X + (int64_t)k0 * 2, LA + ((int64_t)a * rank * K + k0) * 2, low, M, rank, min(kslice, K - k0), nullptr, nullptr,
            nullptr, m0, n0, 0, 0, ring, red, store, K);
        __syncthreads();
    }
}

constexpr int kLowWaves = 8;

// RB: blocks of 16 low-rank values; blockIdx.y takes 16 RB of them.
template <int RB>
__global__ __launch_bounds__(64 * kLowWaves) void lora_low_kernel(const _Float16* __restrict__ X,
                                                                  const _Float16* __restrict__ LA,
                                                                  const int32_t* __restrict__ adapter,
                                                                  const float* __restrict__ lscale, int M, int K,
                                                                  int rank, int rank_p, int adapters,
                                                                  float* __restrict__ low) {
    __shared__ v4f red[kLowWaves * RB * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j16 = lane & 15, g = lane >> 4;
    const int row = blockIdx.x * 16 + j16, r0 = blockIdx.y * 16 * RB;
    int mine = row < M ? adapter[row] : -1;
    if (mine < 0 || mine >= adapters) mine = -1;
    const _Float16* x = X + (int64_t)min(row, M - 1) * K;
    v4f fin[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) fin[b] = v4f{0.f, 0.f, 0.f, 0.f};
    const int tiles = (K + 63) / 64;
    for (uint32_t left = (uint32_t)__builtin_amdgcn_ballot_w64(mine >= 0) & 0xFFFFu; left;) {
        const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
        left &= ~((uint32_t)__builtin_amdgcn_ballot_w64(mine == a) & 0xFFFFu);
        const _Float16* la = LA + (int64_t)a * rank * K;
        v4f cur[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) cur[b] = v4f{0.f, 0.f, 0.f, 0.f};
        auto load = [&](int t, v8h (&xo)[2], v8h (&lo)[RB][2]) __attribute__((always_inline)) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = 64 * t + 32 * s + 8 * g;
                xo[s] = chunk8(x, k, K);
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    lo[b][s] = chunk8(la + (int64_t)min(r0 + 16 * b + j16, rank - 1) * K, k, K);
            }
        };
        v8h xo[2], lo[RB][2];
        if (wave < tiles) load(wave, xo, lo);
        for (int t = wave; t < tiles; t += kLowWaves) {
            v8h xn[2], ln[RB][2];
            if (t + kLowWaves < tiles) load(t + kLowWaves, xn, ln);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    cur[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo[b][s], xo[s], cur[b], 0, 0, 0);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                xo[s] = xn[s];
#pragma unroll
                for (int b = 0; b < RB; ++b) lo[b][s] = ln[b][s];
            }
        }
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) fin[b][e] = mine == a ? cur[b][e] : fin[b][e];
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) red[(wave * RB + b) * 64 + lane] = fin[b];
    __syncthreads();
    const float scale = mine >= 0 ? lscale[mine] : 0.0f;
    for (int b = wave; b < RB; b += kLowWaves) {
        v4f sum = red[b * 64 + lane];
        for (int w = 1; w < kLowWaves; ++w) sum += red[(w * RB + b) * 64 + lane];
        const int r = r0 + 16 * b + 4 * g;
        if (row < M && r < rank_p) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = mine >= 0 && r + e < rank ? sum[e] * scale : 0.0f;
            *reinterpret_cast<v4f*>(low + (int64_t)row * rank_p + r) = sum;
        }
    }
}

constexpr int kLowMostSlices = 8, kLowSliceK = 512;

bool low_ring_ok(const LoraArgs& a) {
    return a.M > kLowDotRows && ring::aligned16(a.X) && ring::aligned16(a.LA) && a.K % 8 == 0 && a.K < (1 << 24);
}

// K of a slice: whole K tiles of the ring kernel.
int64_t low_slice_k(int64_t K, int slices) { return ((K + slices - 1) / slices + 63) / 64 * 64; }

// Rows of one launch: their workgroups (16 rows, up to 512 threads) stay below
// 2^32 threads.
constexpr int64_t kLowLaunchRows = 1 << 24;

hipError_t launch_low_rows(const LoraArgs& a) {
    const _Float16* X = reinterpret_cast<const _Float16*>(a.X);
    const _Float16* LA = reinterpret_cast<const _Float16*>(a.LA);
    const int rank = (int)a.rank, rank_p = (rank + 7) / 8 * 8;
    if (a.M <= kLowDotRows) {
        const int64_t waves = a.M * rank_p;
        lora_low_dot_kernel<<<wide_grid((waves + 3) / 4), 256, 0, a.stream>>>(
            X, LA, a.adapter, a.lscale, waves, (int)a.K, rank, rank_p, (int)a.adapters, a.low);
        return hipGetLastError();
    }
    const unsigned blocks = (unsigned)((a.M + 15) / 16);
    if (low_ring_ok(a)) {
        const unsigned parts = (unsigned)(a.adapters < kLowParts ? a.adapters : kLowParts);
        const unsigned slices = (unsigned)a.low_slices;
        const int kslice = (int)low_slice_k(a.K, a.low_slices);
#define LIBGEMM_GO(BN)                                                                                                \
    lora_low_ring_kernel<BN><<<dim3(blocks, (unsigned)((rank + BN - 1) / BN), parts * slices), 256, 0, a.stream>>>( \
        (const uint8_t*)a.X, (const uint8_t*)a.LA, a.adapter, a.lscale, (int)a.M, (int)a.K, rank, rank_p,           \
        (int)a.adapters, (int)parts, kslice, a.low)
        if (rank <= 16) LIBGEMM_GO(16);
        else if (rank <= 32) LIBGEMM_GO(32);
        else LIBGEMM_GO(64);
#undef LIBGEMM_GO
        return hipGetLastError();
    }
#define LIBGEMM_GO(RB)                                                                                        \
    lora_low_kernel<RB><<<dim3(blocks, (unsigned)((rank + 16 * RB - 1) / (16 * RB))), 64 * kLowWaves, 0, a.stream>>>( \
        X, LA, a.adapter, a.lscale, (int)a.M, (int)a.K, rank, rank_p, (int)a.adapters, a.low)
    if (rank <= 16) LIBGEMM_GO(1);
    else if (rank <= 32) LIBGEMM_GO(2);
    else if (rank <= 64) LIBGEMM_GO(4);
    else LIBGEMM_GO(8);
#undef LIBGEMM_GO
    return hipGetLastError();
}

}  // namespace

// Two workgroups per compute unit, of at least kLowSliceK of K each.
int lora_most_slices(int64_t rows, int64_t rank) {
    if (rows <= kLowDotRows || rank <= 0) return 1;
    const int64_t blocks = (rows + 15) / 16 * ((rank + 63) / 64), s = 512 / blocks;
    return s < 1 ? 1 : (s > kLowMostSlices ? kLowMostSlices : (int)s);
}

int lora_low_slices(const LoraArgs& a) {
    if (!low_ring_ok(a)) return 1;
    const int64_t most = lora_most_slices(a.M, a.rank);
    int64_t s = a.K / kLowSliceK < most ? a.K / kLowSliceK : most;
    if (s <= 1) return 1;
    const int64_t per = low_slice_k(a.K, (int)s);
    return (int)((a.K + per - 1) / per);   // none of them empty
}

hipError_t launch_lora_low(const LoraArgs& call) {
    LoraArgs a = call;
    for (int64_t r0 = 0; r0 < call.M; r0 += kLowLaunchRows) {   // (slices of K: few rows only, one launch)
        a.M = call.M - r0 < kLowLaunchRows ? call.M - r0 : kLowLaunchRows;
        a.X = reinterpret_cast<const _Float16*>(call.X) + r0 * call.K;
        a.adapter = call.adapter + r0;
        a.low = call.low + r0 * ((call.rank + 7) / 8 * 8);
        const hipError_t e = launch_low_rows(a);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace libgemm
