// Register-staged MFMA tile GEMM for gfx950: kernel and launcher templates,
// shared by gemm_tile.hip (configuration table, E4M3 x E4M3 and FP16
// instantiations) and gemm_tile_mixed.hip (the other FP8 operand pairs).
// MFMA tile GEMM for gfx950: C[M,N] = (sA*A[M,K]) (sB*B[K,N]), all row-major.
//
// Operands are FP16 (v_mfma_f32_16x16x32_f16) or OCP E4M3 codes
// (v_mfma_scale_f32_16x16x128_f8f6f4 with neutral block scales), always with
// FP32 accumulation ("DeepGEMM实战：FP8矩阵乘法与JIT编译优化指南" §2.1;
// "HGEMM优化：深度学习中的矩阵乘法性能提升策略" §1.3).
//
// Data flow per workgroup (one BM x BN output tile, 4 waves in a 2 x 2 grid):
//   HBM/L2 --16-byte coalesced loads--> registers --ds_write_b128--> LDS
//   (two LDS stages plus one register stage: tile k+2 is in flight while
//   tile k is multiplied; FP8 guide §2.3 "double buffering", HGEMM §3.2/§3.3
//   on prefetch depth)
//   LDS --ds_read_b128 (A) / ds_read_b64_tr_b16|b8 (B)--> MFMA operands
// A is row-major [M,K]: its K-contiguous rows are exactly the MFMA A operand.
// B is row-major [K,N]: N is contiguous, so the B operand (8 or 32 consecutive
// k for one column per lane) comes from gfx950's LDS transpose reads instead of
// a transposing copy. LDS rows are padded (A: +16 B, B: +16/32 B) so that the
// lanes served by one LDS pass hit distinct banks (the bank-aware layout the
// DeepGEMM deep-dive article, §3.2, argues for).
//
// Edges (FP8 guide §3.3): rows >= M and columns >= N are neither loaded nor
// stored, the K tail is zero-filled in the staged tile, so one kernel serves
// every shape. Interior tiles take a branch-free path; only edge tiles (and
// unaligned operands) run the guarded element loads. The epilogue multiplies
// by sA*sB once and converts to the output type, which is a template
// parameter so that every accumulator index is a compile-time constant and
// the accumulators stay in registers.
//
// Tile order: consecutive workgroups are dispatched round-robin over the 8
// XCDs, each with its own L2. Workgroup ids are remapped so that every XCD
// receives a compact block of tiles (shared A row-blocks and B column-blocks
// stay in one L2), walked in groups of 4 tile rows.

#pragma once

#include "device_common.h"
#include "kernels.h"
#include "tile_order.h"
#include "wide_grid.h"

namespace libgemm {
namespace tile {

// 8-wave kernels with K-major B: read the next A operand before the current
// row block's MFMAs (one more operand register set) and raise the wave's issue
// priority while it issues MFMAs. Measured on one MI355X (us, K-major B):
// E4M3 4096^3 80.2-81.5 -> 78.3, E4M3 16384x12288x4096 822-827 -> 785, FP16
// 4096^3 158-161 -> 151; the same change slowed the row-major kernels (83 ->
// 86, 832 -> 887), whose B operands come from transpose reads, so it is
// applied with K-major B only.
template <bool BT>
constexpr bool kPrefetchA = BT;
template <bool BT>
constexpr bool kMfmaPrio = BT;
// K-major kernels keep A and B rows unpadded (128 bytes) with chunk c of row r
// in slot c ^ ((r >> 1) & 7): the 16 lanes an LDS pass serves (16 consecutive
// rows at one chunk for operand reads, two rows of 8 chunks for the stores)
// then cover all 16 four-bank groups of the 64 banks. Counters on MI355X, per
// 4096^3 launch: FP16 bank-conflict cycles 12.6 M -> 0 (LDS-active 33.6 M ->
// 21.0 M, run time about 1 % lower); FP8, with each lane's operand split over
// chunks g and g + 4 (rd below), 6.3 M -> 0 (LDS-active 16.8 M -> 10.5 M, run
// time 1-2 % lower).
constexpr bool kSwizzleBT = true;

// BT: B is stored K-major, as Bt[N,K] row-major (the layout of a linear
// layer's weight); its tile is then staged and read exactly like A's.
template <int ES, int BM, int BN, int BK, int WM, int WN, bool BT = false>
struct Tile {
    static constexpr int NT = 64 * WM * WN;           // threads per workgroup
    static constexpr int KPI = ES == 2 ? 32 : 128;    // k per MFMA instruction
    static constexpr int OPB = ES == 2 ? 16 : 32;     // operand bytes per lane
    static constexpr int VE = 16 / ES;                // elements per 16-byte chunk
    static constexpr int BKB = BK * ES;               // bytes of one A tile row
    static constexpr int BNB = BN * ES;               // bytes of one B tile row
    static constexpr bool SWZ = BT && kSwizzleBT;     // XOR-swizzled rows (A, and B when K-major)
    static constexpr int SA = SWZ ? BKB : BKB + 16;   // LDS row strides (padded unless swizzled)
    static constexpr int SB = BNB + (ES == 2 ? 32 : 16);
    // B rows come in groups of RB (the rows one 16-lane group of a transpose
    // read spans: 32 for FP8, 8 for FP16) and each group starts 128 bytes
    // further: without that, the row stride times RB is a multiple of the 64
    // banks' 256 bytes and the lane groups that LDS serves together (groups
    // g and g+1 start RB rows apart) read the same 32 banks.
    static constexpr int RB = ES == 2 ? 8 : 32;
    static constexpr int A_BYTES = BM * SA;
    static constexpr int B_BYTES = BT ? BN * SA : BK * SB + (BK / RB) * 128;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int A_CPR = BKB / 16;            // 16-byte chunks per A row
    static constexpr int B_CPR = BT ? BKB / 16 : BNB / 16;
    static constexpr int A_RPP = NT / A_CPR;          // A rows covered per pass of all threads
    static constexpr int B_RPP = NT / B_CPR;
    static constexpr int CA = BM / A_RPP;             // A chunks per thread
    static constexpr int CB = (BT ? BN : BK) / B_RPP;  // B chunks per thread
    static constexpr int WTM = BM / WM, WTN = BN / WN;
    static constexpr int TM = WTM / 16, TN = WTN / 16;
    static constexpr int KS = BK / KPI;
    static_assert(BK % KPI == 0, "BK must be a multiple of the MFMA depth");
    static_assert(NT % A_CPR == 0 && NT % B_CPR == 0, "chunk rows must tile the workgroup");
    static_assert(BM % A_RPP == 0 && (BT ? BN : BK) % B_RPP == 0, "tile chunks must divide evenly");
    static_assert(WTM % 16 == 0 && WTN % 16 == 0, "wave tile must be whole 16x16 blocks");
    static_assert(2 * STAGE <= 160 * 1024, "two stages must fit in LDS");
    static_assert(!SWZ || (A_CPR == 8 && B_CPR == 8 && A_RPP % 16 == 0 && B_RPP % 16 == 0),
                  "the row swizzle assumes 8 chunks per row and row passes of whole 16-row groups");
    // Byte offset of 16-byte chunk c in LDS row r.
    static __device__ __forceinline__ int chunk(int r, int c) { return (SWZ ? (c ^ ((r >> 1) & 7)) : c) * 16; }
    // LDS map: A stage 0, A stage 1, B stage 0, B stage 1
    static constexpr int a_stage(int s) { return s * A_BYTES; }
    static constexpr int b_stage(int s) { return 2 * A_BYTES + s * B_BYTES; }
    // LDS byte offset of staged B row r (a k row, or for BT an n row)
    static __device__ __forceinline__ int b_row(int r) { return BT ? r * SA : r * SB + (r / RB) * 128; }
};

// MFMA operand type, LDS operand reads and the multiply for each element size.
template <int ES>
struct Operand;

template <>
struct Operand<2> {  // FP16: v_mfma_f32_16x16x32_f16, 8 halves per lane
    typedef v8h type;
    template <int FA, int FB>
    static __device__ __forceinline__ v4f mma(v8h a, v8h b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ v8h read_a(const LDS_AS uint8_t* p) {
        return __builtin_bit_cast(v8h, *(const LDS_AS v4u*)p);
    }
    // two transpose reads give k = 8g + 0..3 and 8g + 4..7 of one column
    static __device__ __forceinline__ v8h read_b(const LDS_AS uint8_t* p, int sb) {
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS v4s*)p);
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS v4s*)(p + 4 * sb));
        return __builtin_bit_cast(v8h, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

template <>
struct Operand<1> {  // FP8: v_mfma_scale_f32_16x16x128_f8f6f4 (neutral scales), 32 codes per lane
    typedef v8i type;
    static __device__ __forceinline__ v8i read_a(const LDS_AS uint8_t* p) {
        const v4i lo = *(const LDS_AS v4i*)p;
        const v4i hi = *(const LDS_AS v4i*)(p + 16);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // four transpose reads give k = 32g + 0..7, 8..15, 16..23, 24..31 of one column
    static __device__ __forceinline__ v8i read_b(const LDS_AS uint8_t* p, int sb) {
        const v2i t0 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS_AS v2i*)p);
        const v2i t1 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS_AS v2i*)(p + 8 * sb));
        const v2i t2 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS_AS v2i*)(p + 16 * sb));
        const v2i t3 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS_AS v2i*)(p + 24 * sb));
        const v4i t01 = __builtin_shufflevector(t0, t1, 0, 1, 2, 3);
        const v4i t23 = __builtin_shufflevector(t2, t3, 0, 1, 2, 3);
        return __builtin_shufflevector(t01, t23, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // FA, FB: operand formats (0 = E4M3, 1 = E5M2), the instruction's A and B
    // format selectors.
    template <int FA, int FB>
    static __device__ __forceinline__ v4f mma(v8i a, v8i b, v4f c) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, FA, FB, 0, 127, 0, 127);
    }
};

// One 16-byte chunk of `ES`-byte elements starting at element `col` of a row,
// zero beyond `limit` and for rows out of range (edges and unaligned operands).
template <int ES>
__device__ __forceinline__ v4u load_chunk_guarded(const uint8_t* row_ptr, bool row_ok, int64_t col, int64_t limit) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (row_ok) {
#pragma unroll
        for (int e = 0; e < 16 / ES; ++e) {
            if (col + e < limit) {
                uint32_t v = (ES == 1) ? (uint32_t)row_ptr[col + e]
                                       : (uint32_t)reinterpret_cast<const uint16_t*>(row_ptr)[col + e];
                const int bit = e * ES * 8;
                w[bit >> 5] |= v << (bit & 31);
            }
        }
    }
    return v4u{w[0], w[1], w[2], w[3]};
}

typedef v4u v4u_any __attribute__((aligned(1)));

// load_chunk_guarded for any alignment: a whole chunk is one load; a chunk
// that the row's end cuts is the 16 bytes before that end, shifted down (rows
// shorter than a chunk go element by element).
template <int ES>
__device__ __forceinline__ v4u load_chunk_any(const uint8_t* row_ptr, bool row_ok, int64_t col, int64_t limit) {
    constexpr int VE = 16 / ES;
    if (!row_ok || col >= limit) return v4u{0u, 0u, 0u, 0u};
    if (col + VE <= limit) return *reinterpret_cast<const v4u_any*>(row_ptr + col * ES);
    if (limit < VE) return load_chunk_guarded<ES>(row_ptr, row_ok, col, limit);
    const v4u v = *reinterpret_cast<const v4u_any*>(row_ptr + (limit - VE) * ES);
    const unsigned __int128 w = __builtin_bit_cast(unsigned __int128, v) >> (8 * ES * (int)(col + VE - limit));
    return __builtin_bit_cast(v4u, w);
}

// Eight FP8 codes starting at element col of a row, zero beyond limit and for
// rows out of range.
__device__ __forceinline__ v2i load_codes8_guarded(const uint8_t* row_ptr, bool row_ok, int64_t col, int64_t limit) {
    uint32_t w[2] = {0u, 0u};
    if (row_ok) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < limit) w[e >> 2] |= (uint32_t)row_ptr[col + e] << (8 * (e & 3));
    }
    return v2i{(int)w[0], (int)w[1]};
}

// OUT_E4M3 stands for both FP8 outputs; EPI_E5M2 in eflags (uniform) picks the
// format.
template <int OUT>
__device__ __forceinline__ void store_one(void* C, int64_t idx, float y, int eflags) {
    if constexpr (OUT == OUT_F32) {
        reinterpret_cast<float*>(C)[idx] = y;
    } else if constexpr (OUT == OUT_F16) {
        reinterpret_cast<_Float16*>(C)[idx] = (_Float16)y;
    } else {
        reinterpret_cast<uint8_t*>(C)[idx] = (eflags & EPI_E5M2) ? e5m2_from_f32(y) : e4m3_from_f32(y);
    }
}

// Element k of a row: FP16, or FP8 of format F.
template <int ES, int F>
__device__ __forceinline__ float element(const uint8_t* row, int64_t k) {
    if constexpr (ES == 2) return (float)reinterpret_cast<const _Float16*>(row)[k];
    else if constexpr (F == FMT_E5M2) return __builtin_amdgcn_cvt_f32_bf8((int)row[k], 0);
    else return __builtin_amdgcn_cvt_f32_fp8((int)row[k], 0);
}

// Tiles that the kernels of unaligned operands (UA) hold in registers ahead of
// the LDS, by tile rows. 64: two (over 240 shapes 0.85 to 0.96 of the time with
// one; four, which cost occupancy, 1.01 to 1.05 of that with two).
// 128: one (two take all registers of a second workgroup).
constexpr int kAhead64 = 2, kAhead128 = 1;

// GES: bytes per element of A and B in global memory. GES == ES except for
// the exact FP8 mode (ES = 2, GES = 1): FP8 codes are widened to FP16 as they
// are staged (eflags EPI_A_E5M2 / EPI_B_E5M2 give the operand formats) and
// summed on the FP16 matrix cores.
//
// UA (the products whose weight depends on the row): operands of any element
// alignment keep the vector loads (gfx950's global loads take any address),
// and a row's last partial chunk is read as the 16 bytes that end the row,
// shifted. Ext: what is added to the products before the store (NoExtra, or
// LoraExtra of lora_extra.h), or with kFinish what takes the sums (BiasActExtra of
// bias_act_extra.h).
struct NoExtra {
    static constexpr bool kActive = false, kFinish = false;
};

// One output tile: rows [m0, m0 + BM) below M, columns [n0, n0 + BN) below N,
// K range `split` of kchunk.
template <int ES, int OUT, int BM, int BN, int BK, int WM, int WN, int FA, int FB, bool BT, int GES = ES,
          bool UA = false, class Ext = NoExtra>
__device__ __forceinline__ void tile_body(const uint8_t* __restrict__ A, const uint8_t* __restrict__ B,
                                          void* __restrict__ C, int M, int N, int K, const float* __restrict__ sA,
                                          const float* __restrict__ sB, const float* __restrict__ sOut, int m0, int n0,
                                          int aligned, int eflags, int kchunk, int split, const Ext& ext = Ext{}) {
#include "gemm_tile_body.h"
}

template <int ES, int OUT, int BM, int BN, int BK, int WM, int WN, int FA, int FB, bool BT, int GES = ES,
          bool UA = false, class Ext = NoExtra>
__global__ __launch_bounds__(64 * WM * WN) void gemm_tile_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, void* __restrict__ C, int M, int N, int K,
    const float* __restrict__ sA, const float* __restrict__ sB, const float* __restrict__ sOut, int tiles_m,
    int tiles_n, int aligned, int eflags, int kchunk) {
    int tile_m, tile_n;
    tile_coords(blockIdx.x, tiles_m, tiles_n, tile_m, tile_n);
    const int m0 = tile_m * BM, n0 = tile_n * BN, split = blockIdx.y;
    const Ext ext{};
#include "gemm_tile_body.h"
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Launches one configuration for operand formats FA, FB (FP8 only; FP16 uses
// 0, 0). Defined here for every translation unit that instantiates it.
template <int ES, int BM, int BN, int BK, int WM, int WN, int FA, int FB, bool BT = false, int GES = ES>
hipError_t launch_tile(const GemmArgs& a) {
    const int64_t tiles_m = (a.M + BM - 1) / BM;
    const int64_t tiles_n = (a.N + BN - 1) / BN;
    const int64_t blocks = tiles_m * tiles_n;
    if (blocks <= 0) return hipSuccess;
    if (!launch_holds(blocks, 64 * WM * WN)) return hipErrorInvalidValue;
    const int splits = a.splits > 1 ? a.splits : 1;
    if (splits > 1 && (a.k_chunk % BK != 0 || a.k_chunk <= 0 || (int64_t)(splits - 1) * a.k_chunk >= a.K ||
                       splits > 65535 || !a.ws))
        return hipErrorInvalidValue;
    const int kchunk = splits > 1 ? (int)a.k_chunk : (int)a.K;
    if (BT != (a.b_kmajor != 0)) return hipErrorInvalidValue;
    // Vector loads need 16-byte aligned bases and row pitches (for BT, B's
    // rows are K long like A's, so N needs no alignment).
    // Vector loads read 16 / ES elements: 16 bytes, or 8 bytes of codes when
    // widening.
    const int64_t lb = 16 / ES * GES;
    const bool al = ((uintptr_t)a.A % lb) == 0 && ((uintptr_t)a.B % lb) == 0;
    const int aligned = al && ((a.K * GES) % lb == 0) && (BT || (a.N * GES) % lb == 0);
    const uint8_t* A = reinterpret_cast<const uint8_t*>(a.A);
    const uint8_t* B = reinterpret_cast<const uint8_t*>(a.B);
    const int M = (int)a.M, N = (int)a.N, K = (int)a.K;
    const dim3 grid((unsigned)blocks, (unsigned)splits), block(64 * WM * WN);
    if (splits > 1) {   // FP32 partial sums into the workspace
        const int pflags = EPI_PARTIAL | (GES != ES && a.fmt_a == FMT_E5M2 ? EPI_A_E5M2 : 0) |
                           (GES != ES && a.fmt_b == FMT_E5M2 ? EPI_B_E5M2 : 0);
        gemm_tile_kernel<ES, OUT_F32, BM, BN, BK, WM, WN, FA, FB, BT, GES><<<grid, block, 0, a.stream>>>(
            A, B, a.ws, M, N, K, nullptr, nullptr, nullptr, (int)tiles_m, (int)tiles_n, aligned, pflags, kchunk);
        return hipGetLastError();
    }
    const int eflags = (a.out_dtype == OUT_E5M2 ? EPI_E5M2 : 0) | (a.channel ? EPI_CHANNEL : 0) |
                       (GES != ES && a.fmt_a == FMT_E5M2 ? EPI_A_E5M2 : 0) |
                       (GES != ES && a.fmt_b == FMT_E5M2 ? EPI_B_E5M2 : 0);
    switch (a.out_dtype) {
        case OUT_F32:
            gemm_tile_kernel<ES, OUT_F32, BM, BN, BK, WM, WN, FA, FB, BT, GES><<<grid, block, 0, a.stream>>>(
                A, B, a.C, M, N, K, a.sA, a.sB, a.sOut, (int)tiles_m, (int)tiles_n, aligned, eflags, kchunk);
            break;
        case OUT_F16:
            gemm_tile_kernel<ES, OUT_F16, BM, BN, BK, WM, WN, FA, FB, BT, GES><<<grid, block, 0, a.stream>>>(
                A, B, a.C, M, N, K, a.sA, a.sB, a.sOut, (int)tiles_m, (int)tiles_n, aligned, eflags, kchunk);
            break;
        default:
            if constexpr (GES == 1) {
                gemm_tile_kernel<ES, OUT_E4M3, BM, BN, BK, WM, WN, FA, FB, BT, GES><<<grid, block, 0, a.stream>>>(
                    A, B, a.C, M, N, K, a.sA, a.sB, a.sOut, (int)tiles_m, (int)tiles_n, aligned,
                    eflags, kchunk);
            } else {
                return hipErrorInvalidValue;
            }
    }
    return hipGetLastError();
}

// Operand-format dispatch for configurations compiled for every FP8 pair; the
// pairs other than E4M3 x E4M3 are instantiated in gemm_tile_mixed.hip.
template <int BM, int BN, int BK, int WM, int WN, bool BT = false>
hipError_t launch_tile_fp8_any(const GemmArgs& a) {
    switch (a.fmt_a * 2 + a.fmt_b) {
        case 0: return launch_tile<1, BM, BN, BK, WM, WN, 0, 0, BT>(a);
        case 1: return launch_tile<1, BM, BN, BK, WM, WN, 0, 1, BT>(a);
        case 2: return launch_tile<1, BM, BN, BK, WM, WN, 1, 0, BT>(a);
        default: return launch_tile<1, BM, BN, BK, WM, WN, 1, 1, BT>(a);
    }
}

// The exact-accumulation FP8 mode: FP8 codes in global memory, FP16 in LDS and
// on the matrix cores (formats from the arguments at run time).
template <int BM, int BN, int BK, int WM, int WN, bool BT = false>
hipError_t launch_tile_fp8_exact(const GemmArgs& a) {
    return launch_tile<2, BM, BN, BK, WM, WN, 0, 0, BT, 1>(a);
}

#define LIBGEMM_TILE_MIXED_CONFIGS(X) \
    X(64, 64, 128, 2, 2, false)       \
    X(128, 128, 128, 2, 2, false)     \
    X(256, 256, 128, 2, 4, false)     \
    X(64, 64, 128, 2, 2, true)        \
    X(128, 128, 128, 2, 2, true)      \
    X(256, 256, 128, 2, 4, true)

}  // namespace tile
}  // namespace libgemm
