// Row groups: which rows use which weight, shared by the grouped products.
//
// offsets[G + 1] (device) cuts the rows [0, rows) into G groups; rows before
// offsets[0] and from offsets[G] on belong to no group. The host knows only
// rows and G, so every wave finds its tile itself: the rows form G + 2
// segments (the first and the last belong to no group), segment s has
// ceil(size / BM) rows of tiles, and no tile crosses a segment's end. Offsets
// are clamped to [0, rows]: whatever they hold, no address leaves the operands.
//
// Order. A segment's rows of tiles are cut into equal shares of at most
// kTallest, and a column of a share (those tiles all read one 256-column piece
// of the weight) is what one XCD takes: the columns, counted through all
// segments, go round the 8 XCDs. So each piece of a weight is read into one
// L2, once per share, by tiles that run together; every XCD gets an equal part
// of every group, whatever the groups' sizes; and the rows of A, which all
// XCDs read, are the smaller operand. Consecutive workgroups go round the
// XCDs, so workgroup b takes the (b / 8)th tile of XCD b % 8. (All the groups'
// last, partly filled rows of tiles after all others, to level the load with
// short tiles, measured 5 to 10 % slower: they read the weights again alone.)
// The height of a share hardly matters: shares of up to 3, 6, 12 and 64 rows
// of tiles are within 1 % of each other on 16 to 16384 rows in 8 to 64 groups
// (8192 rows, 8 groups, 4096 x 4096 FP16 280, 281, 281, 281 us; 16384 rows, 16
// groups, 12288 x 4096 FP8 737, 736, 736, 733).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wide_grid.h"

namespace libgemm {

struct RowTile {
    int group;   // -1: rows of no group; -2: no tile left
    int m0;      // first row
    int end;     // end of the segment's rows
    int tn;      // column tile
};

constexpr int kTallest = 6;

// Sum over this lane and those below it (row shifts, then row broadcasts).
__device__ __forceinline__ int wave_running_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// The tile of workgroup bid, the same in every lane of the wave: 64 segments
// at a time, one per lane, running sums for the columns before each segment
// and this XCD's tiles up to it, and a ballot for the segment.
template <int BM>
__device__ __forceinline__ RowTile find_row_tile(const int32_t* __restrict__ offsets, int groups, int rows, int bid,
                                                 int tiles_n) {
    const int lane = threadIdx.x & 63, x = bid & 7;
    int at = bid >> 3;      // tiles of this XCD still to pass over
    int columns = 0;        // of the segments before this 64, modulo 8
    for (int base = 0; base < groups + 2; base += 64) {
        const int s = base + lane;
        int lo = 0, hi = 0;
        if (s <= groups + 1) {
            lo = s == 0 ? 0 : min(max(offsets[s - 1], 0), rows);
            hi = s == groups + 1 ? rows : min(max(offsets[s], 0), rows);
            hi = max(lo, hi);
        }
        const uint32_t tall = ((uint32_t)(hi - lo) + BM - 1) / BM;
        const uint32_t shares = (tall + kTallest - 1) / kTallest;
        const uint32_t low = shares ? tall / shares : 0, more = tall - low * shares;   // `more` shares of low + 1 rows
        const int mine = (int)shares * tiles_n;
        const int upto = wave_running_sum(mine & 7);   // counts modulo 8 place the columns
        const int j0 = (x - columns - upto + (mine & 7)) & 7;   // first column of this XCD
        const int big = (int)more * tiles_n;
        const int n_big = big > j0 ? (big - j0 + 7) >> 3 : 0;
        const int n_all = mine > j0 ? (mine - j0 + 7) >> 3 : 0;
        const int tiles = n_big * (int)(low + 1) + (n_all - n_big) * (int)low;
        const int sum = wave_running_sum(tiles);
        const int here = __builtin_amdgcn_readlane(sum, 63);
        if (at < here) {
            const int l = __popcll(__builtin_amdgcn_ballot_w64(sum <= at));   // the segment's lane
            int i = at - (l ? __builtin_amdgcn_readlane(sum, l - 1) : 0);
            const int q_low = __builtin_amdgcn_readlane((int)low, l), q_more = __builtin_amdgcn_readlane((int)more, l);
            const int q_big = __builtin_amdgcn_readlane(n_big, l);
            int column, row;
            if (i < q_big * (q_low + 1)) {
                column = i / (q_low + 1);
                row = i - column * (q_low + 1);
            } else {
                i -= q_big * (q_low + 1);
                column = i / q_low;
                row = i - column * q_low;
                column += q_big;
            }
            const int j = __builtin_amdgcn_readlane(j0, l) + 8 * column;
            const int share = j / tiles_n;
            row += share * q_low + min(share, q_more);
            const int seg = base + l;
            RowTile r;
            r.group = seg >= 1 && seg <= groups ? seg - 1 : -1;
            r.m0 = __builtin_amdgcn_readlane(lo, l) + row * BM;
            r.end = __builtin_amdgcn_readlane(hi, l);
            r.tn = j - share * tiles_n;
            return r;
        }
        at -= here;
        columns += __builtin_amdgcn_readlane(upto, 63);
    }
    return RowTile{-2, 0, 0, 0};
}

// Workgroups that cover every tile that offsets in order can give: all rows of
// tiles, of which each nonempty segment pads at most one, and for each of them
// its columns rounded up to whole rounds of the XCDs, and one round more. (The
// columns of a share are consecutive numbers, of which one XCD gets at most an
// eighth, rounded up; so the last round is never needed, and those workgroups,
// as those of rows that no segment pads, end after their look at the offsets.)
inline int64_t most_workgroups(int64_t rows, int64_t groups, int bm, int64_t tiles_n) {
    const int64_t segs = groups + 2 < rows ? groups + 2 : rows;
    return (rows + segs * (bm - 1)) / bm * ((tiles_n + 7) / 8 * 8 + 8);
}

// Zeros in columns [n0, n0 + BN) of rows [m0, min(end, m0 + BM)): the rows of no group.
template <int BM, int BN, int ES>
__device__ __forceinline__ void zero_rows(void* C, int m0, int end, int n0, int N) {
    const int rows = min(end - m0, BM), cols = min(N - n0, BN);
    for (int i = threadIdx.x; i < BM * BN; i += blockDim.x) {
        const int r = i / BN, c = i % BN;
        if (r < rows && c < cols) {
            const int64_t at = (int64_t)(m0 + r) * N + n0 + c;
            if (ES == 4) reinterpret_cast<uint32_t*>(C)[at] = 0u;
            else if (ES == 2) reinterpret_cast<uint16_t*>(C)[at] = 0;
            else reinterpret_cast<uint8_t*>(C)[at] = 0;
        }
    }
}

}  // namespace libgemm
