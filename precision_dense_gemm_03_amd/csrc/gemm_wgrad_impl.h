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
// two LDS stages (the layout and padding of gemm_tile_impl.h's row-major B). A step
// takes as long as its one wave per matrix core issues and waits in turn, so the
// loop has no address products, no shifts for rows of whole pieces and no ways out
// (10580 rows, 2304 x 216, 64 x 64: 125 -> 97 us with A in 8 bits; 7240 rows, 128 x
// 3504, FP16: 48 -> 40).
// A product of few tiles is bound by the steps one tile takes one after
// another, so the smaller tile wins there: 1819 rows in 23 groups, 304 x 208:
// 9.5 us with 64, 15.3 with 128, 19.5 ping-pong; 8192 rows in 8 groups, 2048 x
// 4096 into FP32: ping-pong, 164 us, 0.84 PFLOP/s.
//
// One operand may be held as 8-bit values (QS 1: A, 2: B; row_io.h): its codes are
// loaded into registers, two steps ahead, and become FP16 (scaled by the block's
// power of two, rounded to nearest even: exact within FP16's range) as they go to
// the LDS, where everything is as for FP16. offsets may then be NULL: one group. 8192
// rows, 4096 x 4096 into FP32: 214 us with A in 8 bits, 233 with B, 223 with neither.
//
// Order of the tiles: the column tiles of all groups, counted through, go
// round the XCDs, each with all its row tiles, so every XCD gets an equal part
// of every group and tiles that run together share B's columns. A tile takes
// as long as its group has rows, so up to 64 groups come in the order of their
// sizes, the largest first, and the short ones level the end.
#pragma once

#include <cstdlib>
#include <cstring>

#include "gemm_pp_impl.h"
#include "gemm_tile_impl.h"
#include "row_io.h"
#include "wide_grid.h"

namespace libgemm {
namespace {

// An operand of 8-bit values: scales, one byte per 32 columns.
struct MxOperand {
    const uint8_t* scale;
    int64_t blocks;   // scales of a row
};

// Eight codes as FP16, scaled (rounded to nearest even, overflow to infinity; tested
// for every code and scale).
template <int FMT>
__device__ __forceinline__ v4u mx_halves(uint32_t lo, uint32_t hi, float scale) {
    typedef _Float16 v2hh __attribute__((ext_vector_type(2)));
    v4u r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? lo : hi;
        v2hh h;
        if constexpr (FMT == FMT_E5M2)
            h = (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, scale, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, scale, false);
        else
            h = (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, false);
        r[i] = __builtin_bit_cast(uint32_t, h);
    }
    return r;
}

struct WgradTile {
    int group, tm, tn, lo, hi;
};

// The tile of workgroup bid; group -1: none. WHOLE: offsets may be NULL.
template <bool WHOLE>
__device__ __forceinline__ WgradTile wgrad_tile(int bid, const int32_t* __restrict__ offsets, int groups, int rows,
                                                int tiles_m, int tiles_n) {
    const int at = bid >> 3, c = (bid & 7) + 8 * (at / tiles_m);
    WgradTile t{c / tiles_n, at % tiles_m, c % tiles_n, 0, 0};
    if (t.group >= groups) {
        t.group = -1;
        return t;
    }
    if (WHOLE && !offsets) {
        t.hi = rows;
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

// A step's operand reads of the ping-pong kernel with one wait: sixteen of A (four
// blocks of 32 columns at a[i]) and eight of B (two at b[j]), each four rows (2048
// bytes) or sixteen (8192) further. Early-clobber outputs and the wait inside, for the
// reasons given with the groups in device_common.h. Six address registers instead of
// eight new addresses for each of three groups: nothing spills.
__device__ __forceinline__ void wgrad_tr24(v4s (&x)[16], v4s (&y)[8], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %24\n\t"
        "ds_read_b64_tr_b16 %1, %24 offset:2048\n\t"
        "ds_read_b64_tr_b16 %2, %24 offset:8192\n\t"
        "ds_read_b64_tr_b16 %3, %24 offset:10240\n\t"
        "ds_read_b64_tr_b16 %4, %25\n\t"
        "ds_read_b64_tr_b16 %5, %25 offset:2048\n\t"
        "ds_read_b64_tr_b16 %6, %25 offset:8192\n\t"
        "ds_read_b64_tr_b16 %7, %25 offset:10240\n\t"
        "ds_read_b64_tr_b16 %8, %26\n\t"
        "ds_read_b64_tr_b16 %9, %26 offset:2048\n\t"
        "ds_read_b64_tr_b16 %10, %26 offset:8192\n\t"
        "ds_read_b64_tr_b16 %11, %26 offset:10240\n\t"
        "ds_read_b64_tr_b16 %12, %27\n\t"
        "ds_read_b64_tr_b16 %13, %27 offset:2048\n\t"
        "ds_read_b64_tr_b16 %14, %27 offset:8192\n\t"
        "ds_read_b64_tr_b16 %15, %27 offset:10240\n\t"
        "ds_read_b64_tr_b16 %16, %28\n\t"
        "ds_read_b64_tr_b16 %17, %28 offset:2048\n\t"
        "ds_read_b64_tr_b16 %18, %28 offset:8192\n\t"
        "ds_read_b64_tr_b16 %19, %28 offset:10240\n\t"
        "ds_read_b64_tr_b16 %20, %29\n\t"
        "ds_read_b64_tr_b16 %21, %29 offset:2048\n\t"
        "ds_read_b64_tr_b16 %22, %29 offset:8192\n\t"
        "ds_read_b64_tr_b16 %23, %29 offset:10240\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7]), "=&v"(x[8]), "=&v"(x[9]), "=&v"(x[10]), "=&v"(x[11]), "=&v"(x[12]), "=&v"(x[13]), "=&v"(x[14]), "=&v"(x[15]), "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3]), "=&v"(y[4]), "=&v"(y[5]), "=&v"(y[6]), "=&v"(y[7])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b[0]), "v"(b[1])
        : "memory");
}

// LINES: C goes past the caches, in whole 128-byte lines. (A parameter of the
// kernel: of two stores in the branches of a condition the compiler makes one,
// without the hint.)
template <int OUT, bool LINES, int QS = 0, int FMT = 0>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void wgrad_pp_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, void* __restrict__ C,
    const int32_t* __restrict__ offsets, int groups, int rows, int M, int N, int tiles_m, int tiles_n, int vec_out,
    MxOperand mx) {
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
    const WgradTile w = wgrad_tile<QS != 0>((int)wide_block(), offsets, groups, rows, tiles_m, tiles_n);
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

    // ---- 8-bit values: load i of wave j takes rows 8 j + 4 i + lane / 16 of a step, 16
    // codes per lane; two steps in registers. Buffer loads end at the group's last row:
    // codes and scales of rows past it are zeros ----
    const int qr = 8 * wj + (lane >> 4), qc = 2 * (lane & 15);          // row (+ 4 i), first FP16 chunk
    const int qcol = QS ? min(c0 + 8 * qc, W - 16) : 0, qb = (int)mx.blocks;
    const uint8_t* qsrc = (QS == 1 ? A : B) + (QS ? (int64_t)w.lo * W : 0);
    const uint8_t* qscale = QS ? mx.scale + (int64_t)w.lo * qb : nullptr;
    const uint32_t qoff = (uint32_t)(qr * W + qcol), soff = (uint32_t)(qr * qb + qcol / kMxBlock);
    v4u held[2][2];
    uint32_t hscale[2][2];
    auto fetch_via = [&](__amdgpu_buffer_rsrc_t rq, __amdgpu_buffer_rsrc_t rs, int kb, int set) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            held[set][i] = __builtin_amdgcn_raw_buffer_load_b128(rq, qoff, (uint32_t)(kb * BK + 4 * i) * (uint32_t)W, 0);
            hscale[set][i] = __builtin_amdgcn_raw_buffer_load_b8(rs, soff, (uint32_t)(kb * BK + 4 * i) * (uint32_t)qb, 0);
        }
    };
    auto codes_at = [&](int t) __attribute__((always_inline)) {
        return buffer_rsrc(qsrc + (int64_t)t * BK * W, (int64_t)(K - t * BK) * W);
    };
    auto scales_at = [&](int t) __attribute__((always_inline)) {
        return buffer_rsrc(qscale + (int64_t)t * BK * qb, (int64_t)(K - t * BK) * qb);
    };
    // (of a step that may be cut: everything that the bounds check sees in the lane's offset)
    auto fetch = [&](int t, int set) __attribute__((always_inline)) {
        if (t >= nk) return;
        const auto rq = codes_at(t), rs = scales_at(t);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            held[set][i] = __builtin_amdgcn_raw_buffer_load_b128(rq, qoff + (uint32_t)(4 * i) * (uint32_t)W, 0, 0);
            hscale[set][i] = __builtin_amdgcn_raw_buffer_load_b8(rs, soff + (uint32_t)(4 * i) * (uint32_t)qb, 0, 0);
        }
    };
    auto put = [&](int t, int set) __attribute__((always_inline)) {
        LDS_AS uint8_t* dst = QS == 1 ? stage_a(t & 3) : stage_b(t & 3);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const v4u c = held[set][i];
            const float s = mx_scale(hscale[set][i]);
            LDS_AS uint8_t* row = dst + (qr + 4 * i) * 512;
            const int sw = pp::swz_b<2>(qr + 4 * i);
            *(LDS_AS v4u*)(row + ((qc ^ sw) << 4)) = mx_halves<FMT>(c[0], c[1], s);
            *(LDS_AS v4u*)(row + (((qc + 1) ^ sw) << 4)) = mx_halves<FMT>(c[2], c[3], s);
        }
    };

    // ---- operands: transpose reads of rows 16 u + 8 h + 4 q + lane16 / 4,
    // four columns each (gemm_pp_impl.h, row-major B in FP16) ----
    const int lr = lane & 31, h = lane >> 5, j16 = lane & 15, half = (lane >> 4) & 1;
    // (offset in a stage of the read u = q = 0 of the block from column chunk chunk0 on)
    auto addr = [&](int chunk0) __attribute__((always_inline)) -> uint32_t {
        const int k = 8 * h + (j16 >> 2);
        const int chunk = (chunk0 + 2 * half + ((j16 & 3) >> 1)) ^ pp::swz_b<2>(j16 >> 2);
        return (uint32_t)(k * 512 + chunk * 16 + 8 * (j16 & 1));
    };
    uint32_t ra[4], rb[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) ra[i] = addr(16 * G + 4 * i);
#pragma unroll
    for (int j = 0; j < 2; ++j) rb[j] = addr(8 * wj + 4 * j);
    auto pair = [](v4s x, v4s y) __attribute__((always_inline)) -> v8h {
        return __builtin_bit_cast(v8h, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    v8h opa[2][4], opb[2][2];
    auto read = [&](const LDS_AS uint8_t* sa, const LDS_AS uint8_t* sb) __attribute__((always_inline)) {
        v4s x[16], y[8];
        uint32_t aa[4], bb[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) aa[i] = lds_addr(sa) + ra[i];
#pragma unroll
        for (int j = 0; j < 2; ++j) bb[j] = lds_addr(sb) + rb[j];
        wgrad_tr24(x, y, aa, bb);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) opa[u][i] = pair(x[4 * i + 2 * u], x[4 * i + 2 * u + 1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) opb[u][j] = pair(y[4 * j + 2 * u], y[4 * j + 2 * u + 1]);
        }
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
    __amdgpu_buffer_rsrc_t rs_blk, rq_blk;   // (of 8-bit values: rq_blk their codes, rs_blk their scales)
    auto step = [&](auto q, int t, int tmod, bool steady) __attribute__((always_inline)) {
        const int st = steady ? tmod : t & 3;
        read(stage_a(st), stage_b(st));
        if constexpr (decltype(q)::value) {
            // step t + 1 from its registers to the LDS, t + 3 into them
            if (steady) {
                put(tmod + 1, (tmod + 1) & 1);
                fetch_via(rq_blk, rs_blk, tmod + 3, (tmod + 1) & 1);
            } else if (t + 1 < nk) {
                if ((t + 1) & 1) {
                    put(t + 1, 1);
                    fetch(t + 3, 1);
                } else {
                    put(t + 1, 0);
                    fetch(t + 3, 0);
                }
            }
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        } else if (steady) {
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

    auto run = [&](auto q) __attribute__((always_inline)) {
        if constexpr (decltype(q)::value) {
            fetch(0, 0);
            fetch(1, 1);
            put(0, 0);
            fetch(2, 0);
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        } else {
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
        }
        asm volatile("s_barrier" ::: "memory");
        if (G == 1) asm volatile("s_barrier" ::: "memory");
        int t = 0;
        for (; t + 7 <= nk_full; t += 4) {   // loads steps t + 3 .. t + 6
            if constexpr (decltype(q)::value) {
                rq_blk = codes_at(t);
                rs_blk = scales_at(t);
            } else {
                rs_blk = rsrc_at(t);
            }
            step(q, t, 0, true);
            step(q, t + 1, 1, true);
            step(q, t + 2, 2, true);
            step(q, t + 3, 3, true);
        }
#pragma unroll 1
        for (; t < nk; ++t) step(q, t, 0, false);
        if (G == 0) asm volatile("s_barrier" ::: "memory");
    };
    if (nk > 0) {
        if constexpr (QS == 0) run(BoolC<false>{});
        else if (G == QS - 1) run(BoolC<true>{});
        else run(BoolC<false>{});
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

// TS: tile rows and columns, 128 or 64. KG: groups of four waves, each with its own
// LDS stages, that take every KG-th step of 64 rows; their sums meet in the LDS, each
// group storing one of the four blocks of a wave (in a fixed order: results repeat).
template <int OUT, int TS, bool CUT, int QS = 0, int FMT = 0, int KG = 1>
__global__ __launch_bounds__(256 * KG) void wgrad_tile_kernel(const _Float16* __restrict__ A,
                                                         const _Float16* __restrict__ B, void* __restrict__ C,
                                                         const int32_t* __restrict__ offsets, int groups, int rows,
                                                         int M, int N, int tiles_m, int tiles_n, MxOperand mx) {
    using WT = tile::Tile<2, TS, TS, 64, 2, 2, false>;
    constexpr int BK = 64, OP = WT::B_BYTES;   // one operand's stage
    constexpr int CPR = TS / 8, RPP = 256 / CPR, NC = BK / RPP;   // chunks of a row, rows of a pass, passes
    constexpr int WS = TS / 2, TB = TS / 32;   // a wave's rows and columns, in blocks of 16
    constexpr int ST = KG > 1 ? 1 : 2;         // LDS stages (of four groups two each do not fit)
    static_assert(KG == 1 || KG == TB * TB, "a block of a wave for each group");
    __shared__ __attribute__((aligned(16))) uint8_t smem_raw[2 * ST * OP * KG];
    const int kg = KG > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 8) : 0;
    LDS_AS uint8_t* smem = (LDS_AS uint8_t*)smem_raw + 2 * ST * OP * kg;
    const int tid = threadIdx.x & 255, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
    const WgradTile w = wgrad_tile<QS != 0>((int)wide_block(), offsets, groups, rows, tiles_m, tiles_n);
    if (w.group < 0) return;
    const int grp = w.group, m0 = w.tm * TS, n0 = w.tn * TS, lo = w.lo, hi = w.hi;
    const int nk = (hi - lo + BK * KG - 1) / (BK * KG);   // of a group: step kt KG + kg of all

    const int srow = tid / CPR, scol = tid % CPR;   // staged chunk: rows srow + RPP i, 16-byte column scol
    // steps in registers ahead of the LDS (three of sixteen waves' fit); steps unrolled
    constexpr int D = KG > 1 ? 3 : (TS == 64 ? 4 : 1), U = D < 2 ? 2 : D;
    v4u ra[D][NC], rb[D][NC];
    // Loads go out without conditions, in the order of the steps: a lane's pointers go
    // down its rows and stay at the last that the group has, and column chunks past the
    // operand's end are the last whole one (M, N of at least 8); store() clears the one
    // and shifts the other down (CUT: M or N no multiple of 8).
    const int ca = m0 + 8 * scol, cb = n0 + 8 * scol, past_a = ca + 8 - M, past_b = cb + 8 - N;
    const int last = hi - lo - 1;
    constexpr int ESA = QS == 1 ? 1 : 2, ESB = QS == 2 ? 1 : 2;   // bytes of an element
    const uint8_t* pa[NC];
    const uint8_t* pb[NC];
    const uint8_t* ps[NC];   // scales of 8-bit values
    int row[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        row[i] = kg * BK + srow + RPP * i;
        const int64_t r = lo + max(min(row[i], last), 0);
        pa[i] = reinterpret_cast<const uint8_t*>(A) + (r * M + max(min(ca, M - 8), 0)) * ESA;
        pb[i] = reinterpret_cast<const uint8_t*>(B) + (r * N + max(min(cb, N - 8), 0)) * ESB;
        if constexpr (QS != 0) ps[i] = mx.scale + r * mx.blocks + min((QS == 1 ? ca : cb) / kMxBlock, (int)mx.blocks - 1);
    }
    const int64_t step_a = (int64_t)BK * KG * M * ESA, step_b = (int64_t)BK * KG * N * ESB,
                  step_s = (int64_t)BK * KG * mx.blocks;
    // An operand of 8-bit values: eight codes and their scale's byte in a v4u.
    auto load8 = [](const uint8_t* p, const uint8_t* scale) __attribute__((always_inline)) -> v4u {
        const v2u c = *reinterpret_cast<const v2u_b1*>(p);
        return v4u{c[0], c[1], (uint32_t)*scale, 0u};
    };
    auto widened = [](v4u v, int past) __attribute__((always_inline)) -> v4u {
        uint64_t c = (uint64_t)v[0] | ((uint64_t)v[1] << 32);
        if constexpr (CUT) c = past >= 8 ? 0 : (past > 0 ? c >> (8 * past) : c);
        return mx_halves<FMT>((uint32_t)c, (uint32_t)(c >> 32), mx_scale(v[2]));
    };
    auto load = [&](int set) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if constexpr (QS == 1) ra[set][i] = load8(pa[i], ps[i]);
            else ra[set][i] = *reinterpret_cast<const tile::v4u_any*>(pa[i]);
            if constexpr (QS == 2) rb[set][i] = load8(pb[i], ps[i]);
            else rb[set][i] = *reinterpret_cast<const tile::v4u_any*>(pb[i]);
            row[i] += BK * KG;
            const bool more = row[i] <= last;
            pa[i] += more ? step_a : 0;
            pb[i] += more ? step_b : 0;
            if constexpr (QS != 0) ps[i] += more ? step_s : 0;
        }
        // (Loads of two steps mixed before the loop would make every turn of it wait for the
        // newest; so would a way out of its middle.)
        __builtin_amdgcn_sched_barrier(0);
    };
    auto shifted = [](v4u v, int elements) __attribute__((always_inline)) -> v4u {
        if (elements <= 0) return v;
        if (elements >= 8) return v4u{0u, 0u, 0u, 0u};
        return __builtin_bit_cast(v4u, __builtin_bit_cast(unsigned __int128, v) >> (16 * elements));
    };
    auto store = [&](int kt, int st, int set) __attribute__((always_inline)) {
        const int left = last + 1 - (kt * KG + kg) * BK;   // rows of the group from this step on
        v4u a[NC], b[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            a[i] = ra[set][i];
            b[i] = rb[set][i];
            if constexpr (QS == 1) a[i] = widened(a[i], past_a);
            else if constexpr (CUT) a[i] = shifted(a[i], past_a);
            if constexpr (QS == 2) b[i] = widened(b[i], past_b);
            else if constexpr (CUT) b[i] = shifted(b[i], past_b);
        }
        if (left < BK) {
            asm volatile("");   // (a branch: selects would take their time in every step)
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (srow + RPP * i >= left) a[i] = b[i] = v4u{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int at = WT::b_row(srow + RPP * i) + scol * 16;
            *(LDS_AS v4u*)(smem + 2 * st * OP + at) = a[i];
            *(LDS_AS v4u*)(smem + (2 * st + 1) * OP + at) = b[i];
        }
    };
    // (M or N below 8) element by element, straight to the LDS
    auto narrow = [&](int kt) __attribute__((always_inline)) {
#pragma unroll 1
        for (int i = 0; i < NC; ++i) {
            const int r = kt * BK + srow + RPP * i, at = WT::b_row(srow + RPP * i) + scol * 16;
            auto few = [&](const void* base, int c, int width, bool mxv) __attribute__((always_inline)) -> v4u {
                if (!mxv)
                    return tile::load_chunk_any<2>(
                        reinterpret_cast<const uint8_t*>(reinterpret_cast<const _Float16*>(base) + (int64_t)(lo + r) * width),
                        r <= last, c, width);
                uint32_t q[2] = {0u, 0u};
                if (r <= last)
                    for (int e = 0; e < 8 && c + e < width; ++e)
                        q[e / 4] |= (uint32_t)reinterpret_cast<const uint8_t*>(base)[(int64_t)(lo + r) * width + c + e]
                                    << (8 * (e % 4));
                const bool any = r <= last && c < width;
                return mx_halves<FMT>(q[0], q[1],
                                      any ? mx_scale(mx.scale[(int64_t)(lo + r) * mx.blocks + c / kMxBlock]) : 1.0f);
            };
            *(LDS_AS v4u*)(smem + at) = few(A, ca, M, QS == 1);
            *(LDS_AS v4u*)(smem + OP + at) = few(B, cb, N, QS == 2);
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
    if (KG == 1 && (M < 8 || N < 8)) {
#pragma unroll 1
        for (int kt = 0; kt < nk; ++kt) {
            narrow(kt);
            __syncthreads();
            multiply(0);
            __syncthreads();
        }
    } else if (KG > 1 && nk > 0) {
#pragma unroll
        for (int u = 0; u < D; ++u) load(u);
        int k0 = 0;
#pragma unroll 1
        for (; k0 + D <= nk; k0 += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                store(k0 + u, 0, u);
                load(u);
                __syncthreads();
                multiply(0);
                __syncthreads();
            }
        }
#pragma unroll
        for (int u = 0; u < D - 1; ++u) {
            if (k0 + u >= nk) break;
            store(k0 + u, 0, u);
            __syncthreads();
            multiply(0);
            __syncthreads();
        }
    } else if (nk > 0) {
#pragma unroll
        for (int u = 0; u < D; ++u) load(u);
        store(0, 0, 0);
        load(0);
        __syncthreads();
        int k0 = 0;
#pragma unroll 1
        for (; k0 + U < nk; k0 += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {   // step k0 + u, in LDS stage u % 2
                multiply(u & 1);
                store(k0 + u + 1, (u + 1) & 1, (u + 1) % D);
                load((u + 1) % D);
                __syncthreads();
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {   // (loaded already)
            multiply(u & 1);
            if (k0 + u + 1 >= nk) break;
            store(k0 + u + 1, (u + 1) & 1, (u + 1) % D);
            __syncthreads();
        }
    }
    if constexpr (KG > 1) {
        LDS_AS v4f* sums = (LDS_AS v4f*)smem_raw;   // [group][block][256]
#pragma unroll
        for (int b = 0; b < KG; ++b) sums[(kg * KG + b) * 256 + tid] = acc[b / TB][b % TB];
        __syncthreads();
        v4f s = sums[kg * 256 + tid];
#pragma unroll
        for (int q = 1; q < KG; ++q) s += sums[(q * KG + kg) * 256 + tid];
#pragma unroll
        for (int b = 0; b < KG; ++b)
            if (b == kg) acc[b / TB][b % TB] = s;
    }
    const int64_t base = (int64_t)grp * M * N;
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (KG > 1 && i * TB + j != kg) continue;
                const int row = m0 + WS * wm + 16 * i + 4 * g + r, col = n0 + WS * wn + 16 * j + j16;
                if (row < M && col < N) tile::store_one<OUT>(C, base + (int64_t)row * N + col, acc[i][j][r], 0);
            }
}

// Rows and columns of a tile: 256 (the ping-pong kernel), 128 or 64, and 4 for 64 with
// the steps split. qs: the operand of 8-bit values (0: none).
constexpr int kSplit64 = 4;
int choose_wgrad(const GroupedArgs& a, int qs = 0) {
    // 16-byte pieces of both operands' rows, and 32-bit offsets over 8 steps
    const bool pp_ok = pp::aligned16(a.A) && pp::aligned16(a.B) && a.M % (qs == 1 ? 16 : 8) == 0 &&
                       a.N % (qs == 2 ? 16 : 8) == 0 && a.M < (1 << 21) && a.N < (1 << 21);
    // (launches of 1024 threads in a workgroup: far below 2^32 of them)
    const bool split_ok = qs && a.M >= 8 && a.N >= 8 && wgrad_blocks(a.groups, (a.M + 63) / 64, (a.N + 63) / 64) < (1 << 20);
    // Estimated us, fits to measured times of 90 shapes, taken before the tile kernels'
    // loops lost their address products (13 to 17 % of them); with the present kernels
    // choosing by them costs 1.9 % over the fastest of each of 290 further shapes, 20 of
    // which lose more than 10 % (the ping-pong kernel wherever it is possible: 24 % over
    // the 90): tiles over compute units, `more` for the uneven end, no
    // less than `least` for one alone, per_k ns for each of a group's rows, and C
    // stored at no more than tb TB/s.
    struct Cost {
        int size;
        double per_k, least, more, tb, fixed;
    };
    static constexpr Cost f16_costs[] = {{256, 36.8, 0.56, 0.08, 4.8, 9.8},
                                         {128, 14.8, 1.48, 0.04, 3.2, 6.2},
                                         {64, 5.4, 1.50, 0.05, 2.2, 5.6}};
    // With 8-bit values (2100 shapes, 1 to 16384 rows, M and N from 64 to 8192, up to
    // eight groups: 1.7 % over the fastest of each; by the constants above 4.3 %). Splitting
    // the steps pays for few tiles of many rows: 8155 rows, 464 x 72, 38 us for 56; not
    // where tiles fill the chip (3305 rows, 1280 x 656: 45 for 34).
    static constexpr Cost mx_costs[] = {{256, 41.7, 0.545, 0.060, 6.36, 6.98},
                                        {128, 14.7, 1.08, 0.125, 6.37, 6.98},
                                        {64, 4.78, 0.964, 0.307, 5.76, 6.90},
                                        {kSplit64, 8.99, 0.496, 0.013, 1.28, 6.87}};
    int size = 0;
    double least = 0.0;
    const double live = (double)(a.K < a.groups ? (a.K > 0 ? a.K : 1) : a.groups);
    for (int i = 0; i < (qs ? 4 : 3); ++i) {
        const Cost& c = qs ? mx_costs[i] : f16_costs[i];
        if ((c.size == 256 && !pp_ok) || (c.size == kSplit64 && !split_ok)) continue;
        const int side = c.size == kSplit64 ? 64 : c.size;
        const double tiles = (double)a.groups * (double)((a.M + side - 1) / side) * (double)((a.N + side - 1) / side);
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
        if (split_ok && std::strcmp(env, "wgrad_tile_64_split") == 0) size = kSplit64;
    }
    return size;
}

}  // namespace
}  // namespace libgemm
