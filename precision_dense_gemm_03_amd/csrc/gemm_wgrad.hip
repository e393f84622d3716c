// Gradient to the weights of products grouped by rows, for gfx950:
//
//   C[g] = A[rows of g]^T B[rows of g]     A[rows, M], B[rows, N] FP16, C[g] M x N
//
// The sum runs over the group's rows, the slow direction of both operands, so
// both reach the matrix cores through LDS transpose reads (ds_read_b64_tr_b16),
// as row-major B does in the plain products. Rows past the group's end are
// staged as zeros on both sides (another group's rows may hold NaN); a group
// without rows gives zeros. Two kernels, in three tile sizes:
//
// wgrad_pp_kernel (16-byte aligned operands): the ping-pong kernel's plan
// (gemm_pp_impl.h) with A staged like its row-major B. 256 x 256 tiles, 8
// waves in two groups that take turns at the matrix cores and the LDS, 32 rows
// per step (16 KiB of each operand), four LDS stages per operand, direct
// buffer->LDS loads three steps ahead (group 0 loads A, group 1 B).
//
// wgrad_tile_kernel (operands of any alignment): 128 x 128 or 64 x 64 tiles, 4
// waves, 64 rows at a time, one (128) or four (64) steps in registers ahead of
// two LDS stages (the layout and padding of gemm_tile_impl.h's row-major B).
// A product of few tiles is bound by the steps one tile takes one after
// another, so the smaller tile wins there: 1819 rows in 23 groups, 304 x 208:
// 9.5 us with 64, 15.3 with 128, 19.5 ping-pong; 8192 rows in 8 groups, 2048 x
// 4096 into FP32: ping-pong, 164 us, 0.84 PFLOP/s.
//
// Order of the tiles: the column tiles of all groups, counted through, go
// round the XCDs, each with all its row tiles, so every XCD gets an equal part
// of every group and tiles that run together share B's columns. A tile takes
// as long as its group has rows, so up to 64 groups come in the order of their
// sizes, the largest first, and the short ones level the end.
#include <cstdlib>
#include <cstring>

#include "gemm_pp_impl.h"
#include "gemm_tile_impl.h"
#include "wide_grid.h"

namespace libgemm {
namespace {

struct WgradTile {
    int group, tm, tn, lo, hi;
};

// The tile of workgroup bid; group -1: none.
__device__ __forceinline__ WgradTile wgrad_tile(int bid, const int32_t* __restrict__ offsets, int groups, int rows,
                                                int tiles_m, int tiles_n) {
    const int at = bid >> 3, c = (bid & 7) + 8 * (at / tiles_m);
    WgradTile t{c / tiles_n, at % tiles_m, c % tiles_n, 0, 0};
    if (t.group >= groups) {
        t.group = -1;
        return t;
    }
    if (groups <= 64) {
        const int lane = threadIdx.x & 63;
        int size = -1, before = 0;   // groups ahead of this lane's
        if (lane < groups) size = min(max(offsets[lane + 1], 0), rows) - min(max(offsets[lane], 0), rows);
        for (int e = 0; e < groups; ++e) {
            const int other = __builtin_amdgcn_readlane(size, e);
            before += other > size || (other == size && e < lane) ? 1 : 0;
        }
        t.group = __builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < groups && before == t.group));
    }
    t.lo = min(max(offsets[t.group], 0), rows);
    t.hi = max(t.lo, min(max(offsets[t.group + 1], 0), rows));
    return t;
}

int64_t wgrad_blocks(int64_t groups, int64_t tiles_m, int64_t tiles_n) {
    return (groups * tiles_n + 7) / 8 * 8 * tiles_m;
}

// LINES: C goes past the caches, in whole 128-byte lines. (A parameter of the
// kernel: of two stores in the branches of a condition the compiler makes one,
// without the hint.)
template <int OUT, bool LINES>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void wgrad_pp_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, void* __restrict__ C,
    const int32_t* __restrict__ offsets, int groups, int rows, int M, int N, int tiles_m, int tiles_n, int vec_out) {
    constexpr int BK = 32, STAGE = BK * 512, L = 4;   // rows per step, bytes of a stage, loads per wave and step
    __shared__ __attribute__((aligned(1024))) uint8_t a0[STAGE], a1[STAGE], a2[STAGE], a3[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t b0[STAGE], b1[STAGE], b2[STAGE], b3[STAGE];
    auto stage_a = [&](int st) __attribute__((always_inline)) -> LDS_AS uint8_t* {
        switch (st) {
            case 0: return (LDS_AS uint8_t*)a0;
            case 1: return (LDS_AS uint8_t*)a1;
            case 2: return (LDS_AS uint8_t*)a2;
            default: return (LDS_AS uint8_t*)a3;
        }
    };
    auto stage_b = [&](int st) __attribute__((always_inline)) -> LDS_AS uint8_t* {
        switch (st) {
            case 0: return (LDS_AS uint8_t*)b0;
            case 1: return (LDS_AS uint8_t*)b1;
            case 2: return (LDS_AS uint8_t*)b2;
            default: return (LDS_AS uint8_t*)b3;
        }
    };
    const WgradTile w = wgrad_tile((int)wide_block(), offsets, groups, rows, tiles_m, tiles_n);
    if (w.group < 0) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = wave >> 2, wj = wave & 3;
    const int m0 = w.tm * 256, n0 = w.tn * 256;
    const int K = w.hi - w.lo, nk = (K + BK - 1) / BK, nk_full = K / BK;

    // ---- staging: load i of wave j fills rows 2 (4 j + i) and + 1 of a stage
    // (512 bytes each, lane / 32 the row, slot lane % 32 holding chunk
    // slot ^ swz_b(row)); columns past the operand's end read its last chunk ----
    const int W = G == 0 ? M : N, c0 = G == 0 ? m0 : n0;
    const uint8_t* src = (G == 0 ? A : B) + (int64_t)w.lo * W * 2;
    uint32_t off[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int r = 2 * (4 * wj + i) + (lane >> 5);
        const int c = (lane & 31) ^ pp::swz_b<2>(r);
        off[i] = (uint32_t)(r * W + min(c0 + 8 * c, W - 8)) * 2u;
    }
    const uint32_t step_bytes = (uint32_t)BK * (uint32_t)W * 2u;
    const int64_t end = (int64_t)K * W * 2;
    auto rsrc_at = [&](int t) __attribute__((always_inline)) {
        const int64_t at = (int64_t)t * step_bytes;
        return buffer_rsrc(src + at, end - at);
    };
    auto issue_offs = [&](__amdgpu_buffer_rsrc_t rs, const uint32_t (&o)[L], uint32_t kofs, int st)
        __attribute__((always_inline)) {
        if (G == 0) {
            LDS_AS uint8_t* dst = stage_a(st) + wj * 4096;
#pragma unroll
            for (int i = 0; i < L; ++i) buffer_load_lds16(rs, (LDS_AS void*)(dst + i * 1024), o[i], kofs);
        } else {
            LDS_AS uint8_t* dst = stage_b(st) + wj * 4096;
#pragma unroll
            for (int i = 0; i < L; ++i) buffer_load_lds16(rs, (LDS_AS void*)(dst + i * 1024), o[i], kofs);
        }
    };
    auto issue_via = [&](__amdgpu_buffer_rsrc_t rs, int kb, int st) __attribute__((always_inline)) {
        issue_offs(rs, off, (uint32_t)kb * step_bytes, st);
    };
    // The partial last step loads like the others, its rows past the end from
    // the group's last row; clear() puts zeros over those once they have landed.
    auto issue = [&](int t) __attribute__((always_inline)) {
        if (t < nk_full) {
            issue_via(rsrc_at(t), 0, t & 3);
        } else if (t < nk) {
            const int last = K - 1 - t * BK;
            uint32_t o[L];
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int r = 2 * (4 * wj + i) + (lane >> 5);
                o[i] = off[i] - (uint32_t)max(r - last, 0) * (uint32_t)W * 2u;
            }
            issue_offs(rsrc_at(t), o, 0, t & 3);
        }
    };
    auto clear = [&](int t) __attribute__((always_inline)) {
        LDS_AS uint8_t* dst = (G == 0 ? stage_a(t & 3) : stage_b(t & 3)) + wj * 4096;
#pragma unroll
        for (int i = 0; i < L; ++i)
            if (t * BK + 2 * (4 * wj + i) + (lane >> 5) >= K)
                *(LDS_AS v4u*)(dst + i * 1024 + lane * 16) = v4u{0u, 0u, 0u, 0u};
    };

    // ---- operands: transpose reads of rows 16 u + 8 h + 4 q + lane16 / 4,
    // four columns each (gemm_pp_impl.h, row-major B in FP16) ----
    const int lr = lane & 31, h = lane >> 5, j16 = lane & 15, half = (lane >> 4) & 1;
    auto addr = [&](const LDS_AS uint8_t* st, int chunk0, int u, int q) __attribute__((always_inline)) -> uint32_t {
        const int k = 16 * u + 8 * h + 4 * q + (j16 >> 2);
        const int chunk = (chunk0 + 2 * half + ((j16 & 3) >> 1)) ^ pp::swz_b<2>(j16 >> 2);
        return lds_addr(st + k * 512 + chunk * 16 + 8 * (j16 & 1));
    };
    auto pair = [](v4s x, v4s y) __attribute__((always_inline)) -> v8h {
        return __builtin_bit_cast(v8h, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    v8h opa[2][4], opb[2][2];
    auto read = [&](const LDS_AS uint8_t* sa, const LDS_AS uint8_t* sb) __attribute__((always_inline)) {
        v4s t[8];
        uint32_t ad[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) ad[2 * i + q] = addr(sa, 16 * G + 4 * i, u, q);
            lds_tr16_x8(t, ad);
#pragma unroll
            for (int i = 0; i < 4; ++i) opa[u][i] = pair(t[2 * i], t[2 * i + 1]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) ad[4 * u + 2 * j + q] = addr(sb, 8 * wj + 4 * j, u, q);
        lds_tr16_x8(t, ad);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) opb[u][j] = pair(t[4 * u + 2 * j], t[4 * u + 2 * j + 1]);
    };

    v16f acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    // One step: MEM (this group's operand reads, loads three steps ahead, wait
    // for step t + 1's), barrier, MMA, barrier; the other group is one phase off.
    __amdgpu_buffer_rsrc_t rs_blk;
    auto step = [&](int t, int tmod, bool steady) __attribute__((always_inline)) {
        const int st = steady ? tmod : t & 3;
        read(stage_a(st), stage_b(st));
        if (steady) {
            issue_via(rs_blk, tmod + 3, (tmod + 3) & 3);
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * L, 0));
        } else {
            issue(t + 3);
            // step t + 1 must have landed; steps t + 2 and t + 3, where there are any, may be in flight
            if (t + 1 == nk_full && nk > nk_full) {
                __builtin_amdgcn_s_waitcnt(0);
                clear(t + 1);
                __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
            } else if (t + 3 < nk) {
                __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * L, 0));
            } else if (t + 2 < nk) {
                __builtin_amdgcn_s_waitcnt(waitcnt_imm(L, 0));
            } else {
                __builtin_amdgcn_s_waitcnt(0);
            }
        }
        asm volatile("s_barrier" ::: "memory");
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(opa[u][i]));
#pragma unroll
            for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(opb[u][j]));
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(opb[u][j], opa[u][i], acc[i][j], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(acc[i][j]));
        __builtin_amdgcn_s_setprio(0);
        asm volatile("s_barrier" ::: "memory");
    };

    if (nk > 0) {
#pragma unroll
        for (int t = 0; t < 3; ++t) issue(t);
        // step 0 must have landed; steps 1 and 2 may be in flight
        if (nk >= 3) {
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * L, 0));
        } else {
            __builtin_amdgcn_s_waitcnt(0);
            if (nk_full == 0) {
                clear(0);
                __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
            }
        }
        asm volatile("s_barrier" ::: "memory");
        if (G == 1) asm volatile("s_barrier" ::: "memory");
        int t = 0;
        for (; t + 7 <= nk_full; t += 4) {   // loads steps t + 3 .. t + 6
            rs_blk = rsrc_at(t);
            step(t, 0, true);
            step(t + 1, 1, true);
            step(t + 2, 2, true);
            step(t + 3, 3, true);
        }
#pragma unroll 1
        for (; t < nk; ++t) step(t, 0, false);
        if (G == 0) asm volatile("s_barrier" ::: "memory");
    }

    // ---- store: block (i, j), value 4 q + e: row 128 G + 32 i + lr, column
    // 64 wj + 32 j + 8 q + 4 h + e ----
    const int64_t base = (int64_t)w.group * M * N;
    if (!vec_out) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int row = m0 + 128 * G + 32 * i + lr, col = n0 + 64 * wj + 32 * j + 8 * (x >> 2) + 4 * h + (x & 3);
                    if (row < M && col < N) tile::store_one<OUT>(C, base + (int64_t)row * N + col, acc[i][j][x], 0);
                }
        return;
    }
    // Through LDS (a wave's own stage array, free after the last barrier), so
    // that a store writes whole lines of C's rows: 16-byte chunk c of row r sits
    // at slot c ^ (r % chunks of a row). FP32 in two halves of 64 rows.
    constexpr int ES = OUT == OUT_F32 ? 4 : 2, RB = 64 * ES, CH = RB / 16, HALVES = OUT == OUT_F32 ? 2 : 1;
    constexpr int ROWS = 128 / HALVES;
    LDS_AS uint8_t* ep = wave < 4 ? stage_a(wave) : stage_b(wave - 4);
    auto swz = [](int r) __attribute__((always_inline)) -> int { return ES == 4 ? r & 15 : (r >> 1) & 7; };
    uint8_t* Cb = reinterpret_cast<uint8_t*>(C) + base * ES;
#pragma unroll
    for (int half = 0; half < HALVES; ++half) {
#pragma unroll
        for (int ii = 0; ii < 4 / HALVES; ++ii)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = half * (4 / HALVES) + ii, r = 32 * ii + lr;
                    const int cb = (32 * j + 8 * q + 4 * h) * ES;
                    LDS_AS uint8_t* p = ep + r * RB + ((((cb >> 4) ^ swz(r)) << 4) | (cb & 15));
                    if constexpr (OUT == OUT_F32) {
                        *(LDS_AS v4f*)p =
                            v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    } else {
                        typedef _Float16 v4hh __attribute__((ext_vector_type(4)));
                        const v4hh hv = {(_Float16)acc[i][j][4 * q], (_Float16)acc[i][j][4 * q + 1],
                                         (_Float16)acc[i][j][4 * q + 2], (_Float16)acc[i][j][4 * q + 3]};
                        *(LDS_AS v2i*)p = __builtin_bit_cast(v2i, hv);
                    }
                }
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
#pragma unroll
        for (int p = 0; p < ROWS * CH / 64; ++p) {
            const int r = p * (64 / CH) + lane / CH, seg = lane % CH;
            const v4i v = *(const LDS_AS v4i*)(ep + r * RB + 16 * (seg ^ swz(r)));
            const int row = m0 + 128 * G + half * ROWS + r, col = n0 + 64 * wj + seg * (16 / ES);
            if (row < M && col < N) {
                v4i* dst = reinterpret_cast<v4i*>(Cb + ((int64_t)row * N + col) * ES);
                if constexpr (LINES) __builtin_nontemporal_store(v, dst);
                else *dst = v;
            }
        }
    }
}

// TS: tile rows and columns, 128 or 64.
template <int OUT, int TS>
__global__ __launch_bounds__(256) void wgrad_tile_kernel(const _Float16* __restrict__ A,
                                                         const _Float16* __restrict__ B, void* __restrict__ C,
                                                         const int32_t* __restrict__ offsets, int groups, int rows,
                                                         int M, int N, int tiles_m, int tiles_n) {
    using WT = tile::Tile<2, TS, TS, 64, 2, 2, false>;
    constexpr int BK = 64, OP = WT::B_BYTES;   // one operand's stage
    constexpr int CPR = TS / 8, RPP = 256 / CPR, NC = BK / RPP;   // chunks of a row, rows of a pass, passes
    constexpr int WS = TS / 2, TB = TS / 32;   // a wave's rows and columns, in blocks of 16
    __shared__ __attribute__((aligned(16))) uint8_t smem_raw[4 * OP];
    LDS_AS uint8_t* smem = (LDS_AS uint8_t*)smem_raw;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
    const WgradTile w = wgrad_tile((int)wide_block(), offsets, groups, rows, tiles_m, tiles_n);
    if (w.group < 0) return;
    const int grp = w.group, m0 = w.tm * TS, n0 = w.tn * TS, lo = w.lo, hi = w.hi;
    const int nk = (hi - lo + BK - 1) / BK;

    const int srow = tid / CPR, scol = tid % CPR;   // staged chunk: rows srow + RPP i, 16-byte column scol
    constexpr int D = TS == 64 ? 4 : 1, U = D < 2 ? 2 : D;   // steps in registers ahead of the LDS; steps unrolled
    v4u ra[D][NC], rb[D][NC];
    // Loads go out without conditions: rows past the group's end are its last
    // row and column chunks past the operand's end the last whole one (M, N of
    // at least 8); store() clears the one and shifts the other down.
    const int ca = m0 + 8 * scol, cb = n0 + 8 * scol, past_a = ca + 8 - M, past_b = cb + 8 - N;
    const bool cut = (m0 + TS > M && M % 8 != 0) || (n0 + TS > N && N % 8 != 0);
    const _Float16* src_a = A + (int64_t)lo * M + max(min(ca, M - 8), 0);
    const _Float16* src_b = B + (int64_t)lo * N + max(min(cb, N - 8), 0);
    const int last = hi - lo - 1;
    auto load = [&](int kt, int set) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t r = min(kt * BK + srow + RPP * i, last);
            ra[set][i] = *reinterpret_cast<const tile::v4u_any*>(src_a + r * M);
            rb[set][i] = *reinterpret_cast<const tile::v4u_any*>(src_b + r * N);
        }
    };
    auto shifted = [](v4u v, int elements) __attribute__((always_inline)) -> v4u {
        if (elements <= 0) return v;
        if (elements >= 8) return v4u{0u, 0u, 0u, 0u};
        return __builtin_bit_cast(v4u, __builtin_bit_cast(unsigned __int128, v) >> (16 * elements));
    };
    auto store = [&](int kt, int st, int set) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            v4u a = ra[set][i], b = rb[set][i];
            if (cut) {
                a = shifted(a, past_a);
                b = shifted(b, past_b);
            }
            if (kt * BK + srow + RPP * i > last) a = b = v4u{0u, 0u, 0u, 0u};
            const int at = WT::b_row(srow + RPP * i) + scol * 16;
            *(LDS_AS v4u*)(smem + 2 * st * OP + at) = a;
            *(LDS_AS v4u*)(smem + (2 * st + 1) * OP + at) = b;
        }
    };
    // (M or N below 8) element by element, straight to the LDS
    auto narrow = [&](int kt) __attribute__((always_inline)) {
#pragma unroll 1
        for (int i = 0; i < NC; ++i) {
            const int r = kt * BK + srow + RPP * i, at = WT::b_row(srow + RPP * i) + scol * 16;
            const uint8_t* pa = reinterpret_cast<const uint8_t*>(A + (int64_t)(lo + r) * M);
            const uint8_t* pb = reinterpret_cast<const uint8_t*>(B + (int64_t)(lo + r) * N);
            *(LDS_AS v4u*)(smem + at) = tile::load_chunk_any<2>(pa, r <= last, ca, M);
            *(LDS_AS v4u*)(smem + OP + at) = tile::load_chunk_any<2>(pb, r <= last, cb, N);
        }
    };
    const int g = lane >> 4, j16 = lane & 15;
    const int in = WT::b_row(8 * g + (j16 >> 2)) + 8 * (j16 & 3);   // + 2 * column
    v4f acc[TB][TB];
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    auto multiply = [&](int st) __attribute__((always_inline)) {
        const LDS_AS uint8_t* as = smem + 2 * st * OP + in + 2 * WS * wm;
        const LDS_AS uint8_t* bs = smem + (2 * st + 1) * OP + in + 2 * WS * wn;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            v8h bo[TB];
#pragma unroll
            for (int j = 0; j < TB; ++j) bo[j] = tile::Operand<2>::read_b(bs + WT::b_row(32 * ks) + 32 * j, WT::SB);
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                const v8h ao = tile::Operand<2>::read_b(as + WT::b_row(32 * ks) + 32 * i, WT::SB);
#pragma unroll
                for (int j = 0; j < TB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ao, bo[j], acc[i][j], 0, 0, 0);
            }
        }
    };
    if (M < 8 || N < 8) {
#pragma unroll 1
        for (int kt = 0; kt < nk; ++kt) {
            narrow(kt);
            __syncthreads();
            multiply(0);
            __syncthreads();
        }
    } else if (nk > 0) {
#pragma unroll
        for (int u = 0; u < D; ++u) load(u, u);
        store(0, 0, 0);
        load(D, 0);
        __syncthreads();
        for (int k0 = 0; k0 < nk; k0 += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {   // step k0 + u, in LDS stage u % 2
                if (k0 + u >= nk) break;
                multiply(u & 1);
                if (k0 + u + 1 >= nk) break;
                store(k0 + u + 1, (u + 1) & 1, (u + 1) % D);
                load(k0 + u + 1 + D, (u + 1) % D);
                __syncthreads();
            }
        }
    }
    const int64_t base = (int64_t)grp * M * N;
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = m0 + WS * wm + 16 * i + 4 * g + r, col = n0 + WS * wn + 16 * j + j16;
                if (row < M && col < N) tile::store_one<OUT>(C, base + (int64_t)row * N + col, acc[i][j][r], 0);
            }
}

// Rows and columns of a tile: 256 (the ping-pong kernel), 128 or 64.
int choose_wgrad(const GroupedArgs& a) {
    // 16-byte pieces of both operands' rows, and 32-bit offsets over 8 steps
    const bool pp_ok = pp::aligned16(a.A) && pp::aligned16(a.B) && a.M % 8 == 0 && a.N % 8 == 0 &&
                       a.M < (1 << 21) && a.N < (1 << 21);
    // Estimated us, fits to measured times of 90 shapes (choosing by them costs
    // 2 % over the fastest of each shape; the ping-pong kernel wherever it is
    // possible 24 %): tiles over compute units, `more` for the uneven end, no
    // less than `least` for one alone, per_k ns for each of a group's rows, and C
    // stored at no more than tb TB/s.
    struct Cost {
        int size;
        double per_k, least, more, tb, fixed;
    };
    static constexpr Cost costs[] = {{256, 36.8, 0.56, 0.08, 4.8, 9.8},
                                     {128, 14.8, 1.48, 0.04, 3.2, 6.2},
                                     {64, 5.4, 1.50, 0.05, 2.2, 5.6}};
    int size = 0;
    double least = 0.0;
    const double live = (double)(a.K < a.groups ? (a.K > 0 ? a.K : 1) : a.groups);
    for (const Cost& c : costs) {
        if (c.size == 256 && !pp_ok) continue;
        const double tiles = (double)a.groups * (double)((a.M + c.size - 1) / c.size) * (double)((a.N + c.size - 1) / c.size);
        double rounds = tiles / 256.0 + c.more;
        if (rounds < c.least) rounds = c.least;
        const double t = rounds * (double)a.K / live * c.per_k * 1e-3 + c.fixed +
                         (double)a.groups * (double)a.M * (double)a.N * (a.out_dtype == OUT_F32 ? 4.0 : 2.0) / (c.tb * 1e6);
        if (!size || t < least) {
            size = c.size;
            least = t;
        }
    }
    if (const char* env = std::getenv("LIBGEMM_CONFIG")) {
        if (pp_ok && std::strcmp(env, "wgrad_pp") == 0) size = 256;
        if (std::strcmp(env, "wgrad_tile_128") == 0) size = 128;
        if (std::strcmp(env, "wgrad_tile_64") == 0) size = 64;
    }
    return size;
}

}  // namespace

const char* wgrad_kernel_name(const GroupedArgs& a) {
    const int size = choose_wgrad(a);
    return size == 256 ? "wgrad_pp" : (size == 128 ? "wgrad_tile_128" : "wgrad_tile_64");
}

hipError_t launch_grouped_wgrad(const GroupedArgs& a) {
    if (a.M <= 0 || a.N <= 0 || a.groups <= 0) return hipSuccess;
    const int size = choose_wgrad(a);
    const int64_t tiles_m = (a.M + size - 1) / size, tiles_n = (a.N + size - 1) / size;
    const int64_t blocks = wgrad_blocks(a.groups, tiles_m, tiles_n);
    if (blocks > kMostWorkgroups) return hipErrorInvalidValue;
    const dim3 grid = wide_grid(blocks);
    const int rows = (int)a.K, M = (int)a.M, N = (int)a.N, groups = (int)a.groups;
    // Whole lines past the caches: 4096 rows, 8 groups, 2048 x 4096 FP16 102 -> 89
    // us; lines written in two parts, 18 groups of 2232 x 824: 17.9 -> 31.2.
    const bool lines = ((uintptr_t)a.C & 127) == 0 && a.N * (a.out_dtype == OUT_F32 ? 4 : 2) % 128 == 0;
    const int vec_out = pp::aligned16(a.C);
#define LIBGEMM_PP(OUT, LINES)                                                                             \
    wgrad_pp_kernel<OUT, LINES><<<grid, 512, 0, a.stream>>>(                                                \
        (const uint8_t*)a.A, (const uint8_t*)a.B, a.C, a.offsets, groups, rows, M, N, (int)tiles_m,        \
        (int)tiles_n, vec_out)
#define LIBGEMM_TILE(OUT, TS)                                                                                       \
    wgrad_tile_kernel<OUT, TS><<<grid, 256, 0, a.stream>>>((const _Float16*)a.A, (const _Float16*)a.B, \
                                                                       a.C, a.offsets, groups, rows, M, N,          \
                                                                       (int)tiles_m, (int)tiles_n)
    const bool f32 = a.out_dtype == OUT_F32;
    if (size == 256) {
        if (f32 && lines) LIBGEMM_PP(OUT_F32, true);
        else if (f32) LIBGEMM_PP(OUT_F32, false);
        else if (lines) LIBGEMM_PP(OUT_F16, true);
        else LIBGEMM_PP(OUT_F16, false);
    } else if (size == 128) {
        if (f32) LIBGEMM_TILE(OUT_F32, 128);
        else LIBGEMM_TILE(OUT_F16, 128);
    } else {
        if (f32) LIBGEMM_TILE(OUT_F32, 64);
        else LIBGEMM_TILE(OUT_F16, 64);
    }
#undef LIBGEMM_PP
#undef LIBGEMM_TILE
    return hipGetLastError();
}

}  // namespace libgemm
