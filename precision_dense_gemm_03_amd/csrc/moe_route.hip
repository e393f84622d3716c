// Expert routing for gfx950: the k experts of every token, their weights and
// the order of the rows by expert that the grouped products read.
//
//   expert[t, j]  the j-th largest logit's index (equal logits: the lower
//                 index first); -inf and NaN logits are never chosen (-1)
//   weight[t, j]  exp(l_j - top) / sum, the sum over the chosen ones (renorm)
//                 or over all of the token's logits; 0 where expert is -1
//   row[t, j]     the place of (t, j) in the order by (expert, t, j), -1 none
//   offsets[e]    the first row of expert e; token[row] = t, -1 past the last
//
// The order needs, for each (t, j), the number of earlier tokens with the same
// expert. A token chooses an expert at most once, so 64 tokens' choices of an
// expert are one 64-bit word (LDS, set by atomic OR, whose result does not
// depend on order) and that number is a population count of the word's lower
// bits. One workgroup takes a run of 64-token chunks: up to 64 tokens run in
// one launch; beyond, the first launch chooses and leaves each workgroup's
// counts per expert in the workspace, and the second adds the counts of the
// workgroups before it. No atomics on global memory, the same bits each run.
//
// A token is held by 16 lanes (E / 16 logits each, in registers as ordered
// integers); each of the k rounds takes the lanes' largest and reduces it over
// the 16 lanes with row rotations. Bound by that instruction stream and, in the
// second launch, by the wait for the counts: 16384 x 128, k = 8 takes 11.5 and
// 8.5 us, of which reading the 8 MB of logits takes 2; 32 x 64, k = 8 6.4 us in
// its one launch.
#include <hip/hip_runtime.h>
#include <math.h>

#include "moe.h"
#include "wide_grid.h"

namespace libgemm {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024;
constexpr int kChunk = 64;      // tokens per mask word

// Chunks of T tokens (in 64 bits: T may be the largest int).
__host__ __device__ inline int chunks_of(int64_t T) { return (int)((T + kChunk - 1) / kChunk); }

// Total order of the finite and +inf floats as unsigned integers (0: never
// chosen; -0 counts as +0).
__device__ __forceinline__ uint32_t order_of(float v) {
    if (!(v > -INFINITY)) return 0u;   // -inf, NaN
    const uint32_t b = __builtin_bit_cast(uint32_t, v == 0.0f ? 0.0f : v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t o) {
    return __builtin_bit_cast(float, (o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// exp(v - top) with the largest value's own term exactly 1 (+inf included).
__device__ __forceinline__ float exp_below(float v, float top) { return v == top ? 1.0f : expf(v - top); }

template <int ROR>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + ROR, 0xF, 0xF, false);
}

// The larger (order, lower index) pair of this lane's and a rotated lane's;
// idx holds the complement, so that larger means lower.
template <int ROR>
__device__ __forceinline__ void take_larger(uint32_t& ord, uint32_t& idx) {
    const uint32_t o = row_rotate<ROR>(ord), i = row_rotate<ROR>(idx);
    const bool more = o > ord || (o == ord && i > idx);
    ord = more ? o : ord;
    idx = more ? i : idx;
}

// One token on 16 lanes (l = lane % 16): chooses, writes expert and weight and
// sets bit `bit` of the chosen experts' mask words.
template <int VPL>
__device__ __forceinline__ void select_token(const float* __restrict__ lg, int E, int K, bool renorm, int l,
                                             int32_t* __restrict__ expert, float* __restrict__ weight, u64* mask,
                                             int bit) {
    uint32_t ord[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 16 + l;
        ord[i] = e < E ? order_of(lg[e]) : 0u;
    }
    float top = 0.0f, sum = 0.0f, mine[2] = {0.0f, 0.0f};
    int chosen[2] = {-1, -1};
    float all = 0.0f;
    for (int j = 0; j < K; ++j) {
        uint32_t bo = 0u, bi = 0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (ord[i] > bo) {   // the lower index wins within a lane: i ascends
                bo = ord[i];
                bi = ~(uint32_t)(i * 16 + l);
            }
        take_larger<8>(bo, bi);
        take_larger<4>(bo, bi);
        take_larger<2>(bo, bi);
        take_larger<1>(bo, bi);
        if (bo == 0u) break;   // nothing left (the same in all 16 lanes)
        const int e = (int)~bi;
        const float v = value_of(bo);
        if (j == 0) {
            top = v;
            if (!renorm) {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (ord[i]) all += exp_below(value_of(ord[i]), top);
#pragma unroll
                for (int s = 8; s; s >>= 1) all += __shfl_xor(all, s, 16);
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i * 16 + l == e) ord[i] = 0u;
        const float p = exp_below(v, top);
        sum += p;
        if ((j & 15) == l) {
            chosen[j >> 4] = e;
            mine[j >> 4] = p;
            atomicOr(&mask[e], 1ull << bit);
        }
    }
    const float den = renorm ? sum : all;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (h * 16 + l < K) {
            expert[h * 16 + l] = chosen[h];
            weight[h * 16 + l] = chosen[h] >= 0 ? mine[h] / den : 0.0f;
        }
}

// out[e] = sum of in[0 .. e-1] for e <= n (n <= 1024), by all 1024 threads.
__device__ __forceinline__ void exclusive_scan(const int* in, int* out, int n, int* wave_sum) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int v = tid < n ? in[tid] : 0;
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(s, d);
        if (lane >= d) s += u;
    }
    if (lane == 63) wave_sum[w] = s;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < w; ++i) before += wave_sum[i];
    if (tid < n) {
        out[tid] = before + s - v;
        if (tid == n - 1) out[n] = before + s;
    }
    __syncthreads();
}

// Rows of one chunk's choices. base[e]: the next row of expert e; mask: the
// chunk's words when have_mask, else rebuilt from expert[].
__device__ __forceinline__ void assign_chunk(const int32_t* __restrict__ expert, int T, int E, int K, int chunk,
                                             bool have_mask, u64* mask, int* base, int32_t* __restrict__ row,
                                             int32_t* __restrict__ token) {
    const int tid = threadIdx.x;
    const int t0 = chunk * kChunk, n = min(kChunk, T - t0) * K;
    const int64_t at = (int64_t)t0 * K;
    if (!have_mask) {
        for (int e = tid; e < E; e += kThreads) mask[e] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const int e = expert[at + i];
            if (e >= 0) atomicOr(&mask[e], 1ull << (i / K));
        }
        __syncthreads();
    }
    for (int i = tid; i < n; i += kThreads) {
        const int e = expert[at + i], b = i / K;
        int r = -1;
        if (e >= 0) {
            r = base[e] + __popcll(mask[e] & ((1ull << b) - 1));
            token[r] = t0 + b;
        }
        row[at + i] = r;
    }
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) base[e] += __popcll(mask[e]);
    __syncthreads();
}

// Chooses for the chunks of this workgroup. WHOLE (one workgroup): goes on to
// the rows; else its counts per expert go to counts[workgroup, E].
template <int VPL, bool WHOLE>
__global__ __launch_bounds__(kThreads) void route_select_kernel(const float* __restrict__ logits, int T, int E, int K,
                                                                int renorm, int32_t* __restrict__ expert,
                                                                float* __restrict__ weight,
                                                                int32_t* __restrict__ counts, int per_block,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ row,
                                                                int32_t* __restrict__ token) {
    __shared__ u64 mask[VPL * 16];
    __shared__ int cnt[VPL * 16], base[VPL * 16 + 1], wave_sum[kThreads / 64];
    const int tid = threadIdx.x, l = tid & 15;
    const int chunks = chunks_of(T);
    const int c0 = blockIdx.x * per_block, c1 = min(chunks, c0 + per_block);
    for (int e = tid; e < E; e += kThreads) cnt[e] = 0;
    for (int c = c0; c < c1; ++c) {
        for (int e = tid; e < E; e += kThreads) mask[e] = 0;
        __syncthreads();
        const int b = tid >> 4, t = c * kChunk + b;
        if (t < T)
            select_token<VPL>(logits + (int64_t)t * E, E, K, renorm != 0, l, expert + (int64_t)t * K,
                              weight + (int64_t)t * K, mask, b);
        __syncthreads();
        for (int e = tid; e < E; e += kThreads) cnt[e] += __popcll(mask[e]);
        __syncthreads();
    }
    if constexpr (!WHOLE) {
        for (int e = tid; e < E; e += kThreads) counts[(int64_t)blockIdx.x * E + e] = cnt[e];
    } else {
        exclusive_scan(cnt, base, E, wave_sum);
        for (int e = tid; e <= E; e += kThreads) offsets[e] = base[e];
        const int64_t live = base[E];
        __syncthreads();
        for (int64_t i = live + tid; i < (int64_t)T * K; i += kThreads) token[i] = -1;
        for (int c = c0; c < c1; ++c) assign_chunk(expert, T, E, K, c, c1 - c0 == 1, mask, base, row, token);
    }
}

// Rows and tokens from the choices and the workgroups' counts.
__global__ __launch_bounds__(kThreads) void route_assign_kernel(const int32_t* __restrict__ expert,
                                                                const int32_t* __restrict__ counts, int T, int E,
                                                                int K, int per_block, int e_pad,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ row,
                                                                int32_t* __restrict__ token) {
    __shared__ u64 mask[kRouteMaxExperts];
    __shared__ int total[kRouteMaxExperts], before[kRouteMaxExperts], base[kRouteMaxExperts + 1];
    __shared__ int wave_sum[kThreads / 64];
    const int tid = threadIdx.x, blk = blockIdx.x, nblk = gridDim.x;
    for (int e = tid; e < E; e += kThreads) total[e] = before[e] = 0;
    __syncthreads();
    // e_pad: E rounded up to a power of two; kThreads / e_pad threads share an expert
    const int e = tid & (e_pad - 1), part = tid / e_pad, parts = kThreads / e_pad;
    if (e < E) {
        int all = 0, mine = 0;
#pragma unroll 8
        for (int b = part; b < nblk; b += parts) {
            const int c = counts[(int64_t)b * E + e];
            all += c;
            mine += b < blk ? c : 0;
        }
        atomicAdd(&total[e], all);
        atomicAdd(&before[e], mine);
    }
    __syncthreads();
    exclusive_scan(total, base, E, wave_sum);
    const int64_t live = base[E];
    if (blk == 0)
        for (int i = tid; i <= E; i += kThreads) offsets[i] = base[i];
    __syncthreads();
    for (int i = tid; i < E; i += kThreads) base[i] += before[i];
    __syncthreads();
    for (int64_t i = live + (int64_t)blk * kThreads + tid; i < (int64_t)T * K; i += (int64_t)nblk * kThreads)
        token[i] = -1;
    const int chunks = chunks_of(T);
    const int c0 = blk * per_block, c1 = min(chunks, c0 + per_block);
    for (int c = c0; c < c1; ++c) assign_chunk(expert, T, E, K, c, false, mask, base, row, token);
}

// dlogits[t, e]: with S = sum_j w_j dw_j over the chosen experts,
//   renorm      w_j (dw_j - S) at the chosen experts, 0 elsewhere
//   otherwise   p_e ((dw_j where e is chosen, else 0) - S), p the softmax
// One wave per token; the softmax's maximum and sum are taken again from the
// logits (two reads of a row that stays in the L1). 16384 x 128, k = 8: 11.9 us
// with renorm, 15.6 without, for 2.1 and 3.8 us of bytes; the 3 k
// shuffles of each 64 experts are most of its instructions.
__global__ __launch_bounds__(256) void route_backward_kernel(const float* __restrict__ logits,
                                                             const int32_t* __restrict__ expert,
                                                             const float* __restrict__ weight,
                                                             const float* __restrict__ dweight, int T, int E, int K,
                                                             int renorm, float* __restrict__ dlogits) {
    const int lane = threadIdx.x & 63;
    const int64_t t = wide_block() * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const float* lg = logits + t * E;
    int ex = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < K) {
        ex = expert[t * K + lane];
        if (ex >= 0) {
            w = weight[t * K + lane];
            dw = dweight[t * K + lane];
        }
    }
    float S = w * dw;
#pragma unroll
    for (int s = 32; s; s >>= 1) S += __shfl_xor(S, s);
    float top = -INFINITY, sum = 0.0f;
    if (!renorm) {
        for (int e = lane; e < E; e += 64) top = fmaxf(top, lg[e]);   // fmax passes NaN over
#pragma unroll
        for (int s = 32; s; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
        for (int e = lane; e < E; e += 64)
            if (lg[e] > -INFINITY) sum += exp_below(lg[e], top);
#pragma unroll
        for (int s = 32; s; s >>= 1) sum += __shfl_xor(sum, s);
    }
    for (int e0 = 0; e0 < E; e0 += 64) {   // all lanes stay for the shuffles
        const int e = e0 + lane;
        float d = 0.0f, wj = 0.0f;
        for (int j = 0; j < K; ++j) {
            const int xj = __shfl(ex, j);
            const float dj = __shfl(dw, j), pj = __shfl(w, j);
            if (xj == e) {
                d = dj;
                wj = pj;
            }
        }
        if (e < E) {
            float g = 0.0f;
            if (renorm) {
                g = wj != 0.0f ? wj * (d - S) : 0.0f;
            } else if (lg[e] > -INFINITY) {
                g = exp_below(lg[e], top) / sum * (d - S);
            }
            dlogits[t * E + e] = g;
        }
    }
}

template <int VPL>
hipError_t launch_select(const RouteArgs& a, int blocks, int per_block) {
    if (blocks <= 1)
        route_select_kernel<VPL, true><<<1, kThreads, 0, a.stream>>>(
            a.logits, (int)a.T, (int)a.E, (int)a.K, a.renorm, a.expert, a.weight, nullptr, per_block, a.offsets, a.row,
            a.token);
    else
        route_select_kernel<VPL, false><<<blocks, kThreads, 0, a.stream>>>(
            a.logits, (int)a.T, (int)a.E, (int)a.K, a.renorm, a.expert, a.weight, a.counts, per_block, nullptr,
            nullptr, nullptr);
    return hipGetLastError();
}

}  // namespace

int route_blocks(int64_t T, int* per_block) {
    const int chunks = chunks_of(T);
    int blocks = chunks < kRouteMaxBlocks ? chunks : kRouteMaxBlocks;
    if (blocks < 1) blocks = 1;
    const int per = (chunks + blocks - 1) / blocks;
    if (per_block) *per_block = per;
    return per > 0 ? (chunks + per - 1) / per : 1;
}

hipError_t launch_route(const RouteArgs& a) {
    int per = 0;
    const int blocks = route_blocks(a.T, &per);
    hipError_t e;
    if (a.E <= 64) e = launch_select<4>(a, blocks, per);
    else if (a.E <= 128) e = launch_select<8>(a, blocks, per);
    else if (a.E <= 256) e = launch_select<16>(a, blocks, per);
    else if (a.E <= 512) e = launch_select<32>(a, blocks, per);
    else e = launch_select<64>(a, blocks, per);
    if (e != hipSuccess || blocks <= 1) return e;
    int pad = 1;
    while (pad < a.E) pad *= 2;
    route_assign_kernel<<<blocks, kThreads, 0, a.stream>>>(a.expert, a.counts, (int)a.T, (int)a.E, (int)a.K, per, pad,
                                                           a.offsets, a.row, a.token);
    return hipGetLastError();
}

hipError_t launch_route_backward(const float* logits, const int32_t* expert, const float* weight,
                                 const float* dweight, int64_t T, int64_t E, int64_t K, int renorm, float* dlogits,
                                 hipStream_t stream) {
    if (T == 0 || E == 0) return hipSuccess;
    route_backward_kernel<<<wide_grid((T + 3) / 4), 256, 0, stream>>>(logits, expert, weight, dweight, (int)T, (int)E,
                                                                       (int)K, renorm, dlogits);
    return hipGetLastError();
}

}  // namespace libgemm
