// Row groups: which rows use which weight, shared by the grouped products.
//
// offsets[G + 1] (device) cuts the rows [0, rows) into G groups; rows before
// offsets[0] and from offsets[G] on belong to no group. The host knows only
// rows and G, so every wave finds its tile itself: the rows form G + 2
// segments (the first and the last belong to no group), segment s has
// ceil(size / BM) tiles, and a tile's segment comes from a running sum of
// those, 64 segments at a time across the wave's lanes. No tile crosses a
// segment's end. Offsets are clamped to [0, rows]: whatever they hold, no
// address leaves the operands.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libgemm {

struct RowTile {
    int group;   // -1: rows of no group
    int m0;      // first row
    int end;     // end of the segment's rows
};

template <int BM>
struct RowGroups {
    const int32_t* offsets;
    int groups, rows, lane;
    int lo, hi, sum;   // the last scanned 64 segments: this lane's rows, tiles up to and including it
    int total;         // tiles of all segments

    __device__ __forceinline__ int edge(int i) const { return min(max(offsets[i], 0), rows); }

    // Scans segments base .. base + 63; returns their number of tiles.
    __device__ __forceinline__ int scan(int base) {
        const int s = base + lane;
        lo = hi = 0;
        if (s <= groups + 1) {
            lo = s == 0 ? 0 : edge(s - 1);
            hi = s == groups + 1 ? rows : edge(s);
            hi = max(lo, hi);
        }
        sum = (int)(((int64_t)hi - lo + BM - 1) / BM);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(sum, d);
            if (lane >= d) sum += u;
        }
        return __builtin_amdgcn_readlane(sum, 63);
    }

    // limit: the most tiles offsets in order can give (the host's bound).
    __device__ __forceinline__ void init(const int32_t* off, int n, int r, int limit) {
        offsets = off;
        groups = n;
        rows = r;
        lane = threadIdx.x & 63;
        int64_t t = 0;
        for (int base = 0; base < groups + 2; base += 64) t += scan(base);
        total = (int)min(t, (int64_t)limit);
    }

    // The tile tm in [0, total), the same in every lane of the wave.
    __device__ __forceinline__ RowTile find(int tm) {
        int before = 0;
        RowTile r{-1, 0, 0};
        for (int base = 0; base < groups + 2; base += 64) {
            const int here = groups + 2 <= 64 ? __builtin_amdgcn_readlane(sum, 63) : scan(base);
            if (tm < before + here) {
                const int at = __popcll(__builtin_amdgcn_ballot_w64(sum <= tm - before));   // its lane
                const int first = at ? __builtin_amdgcn_readlane(sum, at - 1) : 0;
                const int s = base + at;
                r.group = s >= 1 && s <= groups ? s - 1 : -1;
                r.m0 = __builtin_amdgcn_readlane(lo, at) + (tm - before - first) * BM;
                r.end = __builtin_amdgcn_readlane(hi, at);
                break;
            }
            before += here;
        }
        return r;
    }
};

// The most tiles of BM rows that G groups in order can give: each nonempty
// segment adds at most BM - 1 padded rows.
inline int64_t most_row_tiles(int64_t rows, int64_t groups, int bm) {
    const int64_t segs = groups + 2 < rows ? groups + 2 : rows;
    return (rows + segs * (bm - 1)) / bm;
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
