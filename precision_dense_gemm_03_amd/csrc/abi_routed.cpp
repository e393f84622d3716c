// C-ABI entry points of the products whose weight depends on the row (grouped
// by expert, per-row adapters) and of expert routing (include/libgemm.h).
// Arguments are validated before any HIP call, as in abi.cpp.
#include "abi_common.h"
#include "kernels.h"
#include "moe.h"

using namespace libgemm;

namespace {

int run_grouped(int kind, const GroupedArgs& a) {
    const int st = check_device();
    if (st != GEMM_OK) return st;
    if (a.K == 0 || a.groups == 0) return status_of(launch_fill_zero(a.C, a.M * a.N, a.out_dtype, a.stream));
    return status_of(launch_grouped(kind, a));
}

int grouped_common(int kind, const void* A, int fmt_a, const void* B, int fmt_b, const int32_t* offsets,
                   const float* sA, const float* sB, const float* sOut, void* C, int out_dtype, int64_t rows, int64_t N,
                   int64_t K, int64_t groups, int channel, int b_kmajor, hipStream_t stream) {
    const int64_t es = kind == KIND_F16 ? 2 : 1;
    if (out_dtype < GEMM_OUT_F32 || out_dtype > (kind == KIND_F16 ? GEMM_OUT_F16 : GEMM_OUT_E5M2)) return GEMM_ERR_DTYPE;
    if (!fmt_ok(fmt_a) || !fmt_ok(fmt_b)) return GEMM_ERR_DTYPE;
    const int64_t os = out_size(out_dtype);
    if (!size_ok(rows) || !size_ok(N) || !size_ok(K) || groups < 0 || groups > kMaxRowGroups) return GEMM_ERR_DIM;
    if (!bytes_ok(rows, K, es) || !bytes_ok(rows, N, os) || !bytes3_ok(K, N, groups, es)) return GEMM_ERR_DIM;
    if (rows == 0 || N == 0) return GEMM_OK;
    if (!C || !offsets) return GEMM_ERR_NULL;
    const bool reads = K > 0 && groups > 0;
    if (reads && (!A || !B)) return GEMM_ERR_NULL;
    if (kind == KIND_FP8 && (!sA || (groups > 0 && !sB))) return GEMM_ERR_NULL;
    if (fp8_out(out_dtype) && !sOut) return GEMM_ERR_SCALE;
    const Range w[1] = {{C, rows * N * os}};
    const Range r[6] = {{A, reads ? rows * K * es : 0}, {B, reads ? groups * K * N * es : 0},
                        {offsets, 4 * (groups + 1)}, {sA, kind == KIND_FP8 ? (channel ? 4 * rows : 4) : 0},
                        {sB, kind == KIND_FP8 ? (channel ? 4 * groups * N : 4 * groups) : 0},
                        {sOut, fp8_out(out_dtype) ? 4 : 0}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    GroupedArgs a;
    static_cast<GemmArgs&>(a) = GemmArgs{A, B, C, sA, sB, fp8_out(out_dtype) ? sOut : nullptr, out_dtype, rows, N, K,
                                         stream, fmt_a, fmt_b, channel};
    a.b_kmajor = b_kmajor;
    a.offsets = offsets;
    a.groups = groups;
    return run_grouped(kind, a);
}

int64_t lora_low_bytes(int64_t rows, int64_t rank) {
    return lora_most_slices(rows, rank) * rows * ((rank + 7) / 8 * 8) * 4;
}

int lora_common(int kind, const void* A, int fmt_a, const void* Bt, int fmt_b, const float* sA, const float* sB,
                const void* X, const void* LA, const void* LB, const int32_t* adapter, const float* lscale, void* C,
                int out_dtype, int64_t rows, int64_t N, int64_t K, int64_t rank, int64_t adapters, void* ws,
                int64_t ws_bytes, hipStream_t stream) {
    const int64_t es = kind == KIND_F16 ? 2 : 1;
    if (out_dtype != GEMM_OUT_F32 && out_dtype != GEMM_OUT_F16) return GEMM_ERR_DTYPE;
    if (!fmt_ok(fmt_a) || !fmt_ok(fmt_b)) return GEMM_ERR_DTYPE;
    const int64_t os = out_size(out_dtype);
    if (!size_ok(rows) || !size_ok(N) || !size_ok(K) || !size_ok(rank) || !dim_ok(adapters)) return GEMM_ERR_DIM;
    if (!bytes_ok(rows, K, 2) || !bytes_ok(K, N, es) || !bytes_ok(rows, N, os) || !bytes3_ok(rank, K, adapters, 2) ||
        !bytes3_ok(rank, N, adapters, 2) || !bytes_ok(rows, rank + 7, 32))
        return GEMM_ERR_DIM;
    if (rows == 0 || N == 0) return GEMM_OK;
    if (!C) return GEMM_ERR_NULL;
    const bool low = rank > 0 && adapters > 0 && K > 0;
    if (K > 0 && (!A || !Bt)) return GEMM_ERR_NULL;
    if (kind == KIND_FP8 && (!sA || !sB)) return GEMM_ERR_NULL;
    if (low && (!X || !LA || !LB || !adapter || !lscale || !ws)) return GEMM_ERR_NULL;
    const int64_t need = low ? lora_low_bytes(rows, rank) : 0;
    if (low && (ws_bytes < need || ((uintptr_t)ws & 15u) != 0)) return GEMM_ERR_WORKSPACE;
    const Range w[2] = {{C, rows * N * os}, {ws, need}};
    const Range r[9] = {{A, rows * K * es}, {Bt, K * N * es}, {sA, kind == KIND_FP8 ? 4 * rows : 0},
                        {sB, kind == KIND_FP8 ? 4 * N : 0}, {X, low ? rows * K * 2 : 0},
                        {LA, low ? adapters * rank * K * 2 : 0}, {LB, low ? adapters * rank * N * 2 : 0},
                        {adapter, low ? 4 * rows : 0}, {lscale, low ? 4 * adapters : 0}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    LoraArgs a;
    static_cast<GemmArgs&>(a) = GemmArgs{A, Bt, C, sA, sB, nullptr, out_dtype, rows, N, K, stream, fmt_a, fmt_b,
                                         kind == KIND_FP8 ? 1 : 0};
    a.b_kmajor = 1;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    if (K == 0) return status_of(launch_fill_zero(C, rows * N, out_dtype, stream));
    if (!low) {   // no adapter at all: the plain product
        const GemmConfig* cfg = select_config(kind, out_dtype, rows, N, K, fmt_a, fmt_b, 1);
        return cfg ? status_of(cfg->launch(a)) : GEMM_ERR_UNSUPPORTED;
    }
    a.X = X;
    a.LA = LA;
    a.LB = LB;
    a.adapter = adapter;
    a.lscale = lscale;
    a.rank = rank;
    a.adapters = adapters;
    a.low = reinterpret_cast<float*>(ws);
    return status_of(launch_lora(kind, a));
}

}  // namespace

extern "C" {

int gemm_f16_grouped(const void* A, const void* B, const int32_t* offsets, void* C, int out_dtype, int64_t rows,
                     int64_t N, int64_t K, int64_t groups, hipStream_t stream) {
    return grouped_common(KIND_F16, A, 0, B, 0, offsets, nullptr, nullptr, nullptr, C, out_dtype, rows, N, K, groups, 0,
                          0, stream);
}

int gemm_f16_grouped_bt(const void* A, const void* Bt, const int32_t* offsets, void* C, int out_dtype, int64_t rows,
                        int64_t N, int64_t K, int64_t groups, hipStream_t stream) {
    return grouped_common(KIND_F16, A, 0, Bt, 0, offsets, nullptr, nullptr, nullptr, C, out_dtype, rows, N, K, groups,
                          0, 1, stream);
}

int gemm_fp8_grouped(const uint8_t* A, int fmt_a, const uint8_t* B, int fmt_b, const int32_t* offsets, const float* sA,
                     const float* sB, const float* sOut, void* C, int out_dtype, int64_t rows, int64_t N, int64_t K,
                     int64_t groups, hipStream_t stream) {
    return grouped_common(KIND_FP8, A, fmt_a, B, fmt_b, offsets, sA, sB, sOut, C, out_dtype, rows, N, K, groups, 0, 0,
                          stream);
}

int gemm_fp8_grouped_bt(const uint8_t* A, int fmt_a, const uint8_t* Bt, int fmt_b, const int32_t* offsets,
                        const float* sA, const float* sB, const float* sOut, void* C, int out_dtype, int64_t rows,
                        int64_t N, int64_t K, int64_t groups, hipStream_t stream) {
    return grouped_common(KIND_FP8, A, fmt_a, Bt, fmt_b, offsets, sA, sB, sOut, C, out_dtype, rows, N, K, groups, 0, 1,
                          stream);
}

int gemm_fp8_grouped_channel(const uint8_t* A, int fmt_a, const uint8_t* B, int fmt_b, const int32_t* offsets,
                             const float* sA, const float* sB, const float* sOut, void* C, int out_dtype, int64_t rows,
                             int64_t N, int64_t K, int64_t groups, hipStream_t stream) {
    return grouped_common(KIND_FP8, A, fmt_a, B, fmt_b, offsets, sA, sB, sOut, C, out_dtype, rows, N, K, groups, 1, 0,
                          stream);
}

int gemm_fp8_grouped_channel_bt(const uint8_t* A, int fmt_a, const uint8_t* Bt, int fmt_b, const int32_t* offsets,
                                const float* sA, const float* sB, const float* sOut, void* C, int out_dtype,
                                int64_t rows, int64_t N, int64_t K, int64_t groups, hipStream_t stream) {
    return grouped_common(KIND_FP8, A, fmt_a, Bt, fmt_b, offsets, sA, sB, sOut, C, out_dtype, rows, N, K, groups, 1, 1,
                          stream);
}

int gemm_f16_grouped_wgrad(const void* A, const void* B, const int32_t* offsets, void* C, int out_dtype, int64_t rows,
                           int64_t M, int64_t N, int64_t groups, hipStream_t stream) {
    if (out_dtype != GEMM_OUT_F32 && out_dtype != GEMM_OUT_F16) return GEMM_ERR_DTYPE;
    const int64_t os = out_size(out_dtype);
    if (!size_ok(rows) || !size_ok(M) || !size_ok(N) || groups < 0 || groups > kMaxRowGroups) return GEMM_ERR_DIM;
    if (!bytes_ok(rows, M, 2) || !bytes_ok(rows, N, 2) || !bytes3_ok(M, N, groups, os)) return GEMM_ERR_DIM;
    if (M == 0 || N == 0 || groups == 0) return GEMM_OK;
    if (!C || !offsets || (rows > 0 && (!A || !B))) return GEMM_ERR_NULL;
    const Range w[1] = {{C, groups * M * N * os}};
    const Range r[3] = {{A, rows * M * 2}, {B, rows * N * 2}, {offsets, 4 * (groups + 1)}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    GroupedArgs a;
    static_cast<GemmArgs&>(a) = GemmArgs{A, B, C, nullptr, nullptr, nullptr, out_dtype, M, N, rows, stream};
    a.offsets = offsets;
    a.groups = groups;
    return status_of(launch_grouped_wgrad(a));
}

int64_t gemm_lora_workspace_size(int64_t rows, int64_t rank) {
    if (!size_ok(rows) || !size_ok(rank) || !bytes_ok(rows, rank + 7, 32)) return GEMM_ERR_DIM;
    return lora_low_bytes(rows, rank);
}

int gemm_f16_lora_bt(const void* A, const void* Bt, const void* LA, const void* LB, const int32_t* adapter,
                     const float* lscale, void* C, int out_dtype, int64_t rows, int64_t N, int64_t K, int64_t rank,
                     int64_t adapters, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    return lora_common(KIND_F16, A, 0, Bt, 0, nullptr, nullptr, A, LA, LB, adapter, lscale, C, out_dtype, rows, N, K,
                       rank, adapters, workspace, workspace_bytes, stream);
}

int gemm_fp8_lora_bt(const uint8_t* A, int fmt_a, const uint8_t* Bt, int fmt_b, const float* sA, const float* sB,
                     const void* X, const void* LA, const void* LB, const int32_t* adapter, const float* lscale,
                     void* C, int out_dtype, int64_t rows, int64_t N, int64_t K, int64_t rank, int64_t adapters,
                     void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    return lora_common(KIND_FP8, A, fmt_a, Bt, fmt_b, sA, sB, X, LA, LB, adapter, lscale, C, out_dtype, rows, N, K,
                       rank, adapters, workspace, workspace_bytes, stream);
}

static bool kinds_ok(int kind, int out_dtype, int most_out, int fmt_a, int fmt_b) {
    if (kind != KIND_F16 && kind != KIND_FP8) return false;
    if (out_dtype < GEMM_OUT_F32 || out_dtype > (kind == KIND_F16 ? GEMM_OUT_F16 : most_out)) return false;
    return fmt_ok(fmt_a) && fmt_ok(fmt_b);
}

int gemm_select_config_grouped(int kind, int out_dtype, int64_t rows, int64_t N, int64_t K, int64_t groups, int fmt_a,
                               int fmt_b, int b_kmajor, char* buf, int buflen) {
    if (!kinds_ok(kind, out_dtype, GEMM_OUT_E5M2, fmt_a, fmt_b)) return GEMM_ERR_DTYPE;
    if (!size_ok(rows) || !size_ok(N) || !size_ok(K) || groups < 0 || groups > kMaxRowGroups) return GEMM_ERR_DIM;
    GroupedArgs a;
    static_cast<GemmArgs&>(a) = GemmArgs{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, out_dtype, rows, N, K,
                                         nullptr, kind == KIND_F16 ? 0 : fmt_a, kind == KIND_F16 ? 0 : fmt_b, 0};
    a.b_kmajor = b_kmajor ? 1 : 0;
    a.groups = groups;
    return put_name(grouped_kernel_name(kind, a), buf, buflen);
}

int gemm_select_config_wgrad(int out_dtype, int64_t rows, int64_t M, int64_t N, int64_t groups, char* buf, int buflen) {
    if (out_dtype != GEMM_OUT_F32 && out_dtype != GEMM_OUT_F16) return GEMM_ERR_DTYPE;
    if (!size_ok(rows) || !size_ok(M) || !size_ok(N) || groups < 0 || groups > kMaxRowGroups) return GEMM_ERR_DIM;
    GroupedArgs a;
    static_cast<GemmArgs&>(a) = GemmArgs{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, out_dtype, M, N, rows,
                                         nullptr};
    a.groups = groups;
    return put_name(wgrad_kernel_name(a), buf, buflen);
}

int gemm_select_config_lora(int kind, int out_dtype, int64_t rows, int64_t N, int64_t K, int64_t rank, int64_t adapters,
                            int fmt_a, int fmt_b, char* buf, int buflen) {
    if (!kinds_ok(kind, out_dtype, GEMM_OUT_F16, fmt_a, fmt_b)) return GEMM_ERR_DTYPE;
    if (!size_ok(rows) || !size_ok(N) || !size_ok(K) || !size_ok(rank) || !dim_ok(adapters)) return GEMM_ERR_DIM;
    LoraArgs a;
    static_cast<GemmArgs&>(a) = GemmArgs{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, out_dtype, rows, N, K,
                                         nullptr, kind == KIND_F16 ? 0 : fmt_a, kind == KIND_F16 ? 0 : fmt_b, 0};
    a.b_kmajor = 1;
    a.rank = rank;
    a.adapters = adapters;
    return put_name(lora_kernel_name(kind, a), buf, buflen);
}

// ------------------------------------------------------------- expert routing

static bool route_dims_ok(int64_t T, int64_t E, int64_t K) {
    return dim_ok(T) && E >= 1 && E <= kRouteMaxExperts && K >= 1 && K <= kRouteMaxTopk && K <= E &&
           T * K <= kMaxDim;
}

int64_t moe_route_workspace_size(int64_t tokens, int64_t experts) {
    if (!dim_ok(tokens) || experts < 1 || experts > kRouteMaxExperts) return GEMM_ERR_DIM;
    const int64_t blocks = route_blocks(tokens);
    return blocks > 1 ? blocks * experts * 4 : 0;
}

int moe_route_f32(const float* logits, int64_t tokens, int64_t experts, int64_t topk, int renorm, int32_t* expert,
                  float* weight, int32_t* offsets, int32_t* row, int32_t* token, void* workspace,
                  int64_t workspace_bytes, hipStream_t stream) {
    if (!route_dims_ok(tokens, experts, topk)) return GEMM_ERR_DIM;
    if (!offsets) return GEMM_ERR_NULL;
    if (tokens > 0 && (!logits || !expert || !weight || !row || !token)) return GEMM_ERR_NULL;
    const int64_t need = moe_route_workspace_size(tokens, experts);
    if (need > 0) {
        if (!workspace) return GEMM_ERR_NULL;
        if (workspace_bytes < need || ((uintptr_t)workspace & 15u) != 0) return GEMM_ERR_WORKSPACE;
    }
    const int64_t n = 4 * tokens * topk;
    const Range w[6] = {{expert, n}, {weight, n}, {offsets, 4 * (experts + 1)}, {row, n}, {token, n}, {workspace, need}};
    const Range r[1] = {{logits, 4 * tokens * experts}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    return status_of(launch_route(RouteArgs{logits, tokens, experts, topk, renorm ? 1 : 0, expert, weight, offsets, row,
                                            token, reinterpret_cast<int32_t*>(workspace), stream}));
}

int moe_route_backward_f32(const float* logits, const int32_t* expert, const float* weight, const float* dweight,
                           int64_t tokens, int64_t experts, int64_t topk, int renorm, float* dlogits,
                           hipStream_t stream) {
    if (!route_dims_ok(tokens, experts, topk)) return GEMM_ERR_DIM;
    if (tokens == 0) return GEMM_OK;
    if (!logits || !expert || !weight || !dweight || !dlogits) return GEMM_ERR_NULL;
    const int64_t n = 4 * tokens * topk, l = 4 * tokens * experts;
    const Range w[1] = {{dlogits, l}};
    const Range r[4] = {{logits, l}, {expert, n}, {weight, n}, {dweight, n}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    return status_of(launch_route_backward(logits, expert, weight, dweight, tokens, experts, topk, renorm ? 1 : 0,
                                           dlogits, stream));
}

int moe_gather(const void* x, const int32_t* token, void* y, int64_t tokens, int64_t rows, int64_t width,
               int elem_bytes, hipStream_t stream) {
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return GEMM_ERR_DTYPE;
    if (!dim_ok(tokens) || !dim_ok(rows) || !dim_ok(width) || !bytes_ok(tokens, width, elem_bytes) ||
        !bytes_ok(rows, width, elem_bytes))
        return GEMM_ERR_DIM;
    if (rows == 0 || width == 0) return GEMM_OK;
    if (!token || !y || (tokens > 0 && !x)) return GEMM_ERR_NULL;
    const Range w[1] = {{y, rows * width * elem_bytes}};
    const Range r[2] = {{x, tokens * width * elem_bytes}, {token, 4 * rows}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    return status_of(launch_moe_gather(x, token, y, tokens, rows, width * elem_bytes, stream));
}

static bool float_type(int t) { return t == GEMM_OUT_F32 || t == GEMM_OUT_F16; }

int moe_combine(const void* z, int z_dtype, const int32_t* row, const float* weight, void* y, int y_dtype,
                int64_t tokens, int64_t topk, int64_t rows, int64_t width, hipStream_t stream) {
    if (!float_type(z_dtype) || !float_type(y_dtype)) return GEMM_ERR_DTYPE;
    if (!dim_ok(tokens) || topk < 1 || topk > kRouteMaxTopk || !dim_ok(rows) || !dim_ok(width) ||
        tokens * topk > kMaxDim || !bytes_ok(tokens, width, 4) || !bytes_ok(rows, width, 4))
        return GEMM_ERR_DIM;
    if (tokens == 0 || width == 0) return GEMM_OK;
    if (!row || !y || (rows > 0 && !z)) return GEMM_ERR_NULL;
    const Range w[1] = {{y, tokens * width * out_size(y_dtype)}};
    const Range r[3] = {{z, rows * width * out_size(z_dtype)}, {row, 4 * tokens * topk}, {weight, 4 * tokens * topk}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    return status_of(launch_moe_combine(z, z_dtype, row, weight, y, y_dtype, tokens, topk, rows, width, stream));
}

int moe_combine_backward(const void* dy, const void* z, int dtype, const int32_t* row, const float* weight, void* dz,
                         float* dweight, int64_t tokens, int64_t topk, int64_t rows, int64_t width,
                         hipStream_t stream) {
    if (!float_type(dtype)) return GEMM_ERR_DTYPE;
    if (!dim_ok(tokens) || topk < 1 || topk > kRouteMaxTopk || !dim_ok(rows) || !dim_ok(width) ||
        tokens * topk > kMaxDim || !bytes_ok(tokens, width, 4) || !bytes_ok(rows, width, 4))
        return GEMM_ERR_DIM;
    if (tokens == 0) return GEMM_OK;
    if (!row || !weight || !dweight) return GEMM_ERR_NULL;
    if (width > 0 && (!dy || (rows > 0 && (!z || !dz)))) return GEMM_ERR_NULL;
    const int64_t es = out_size(dtype), n = 4 * tokens * topk;
    const Range w[2] = {{dz, rows * width * es}, {dweight, n}};
    const Range r[4] = {{dy, tokens * width * es}, {z, rows * width * es}, {row, n}, {weight, n}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    return status_of(launch_moe_combine_backward(dy, z, dtype, row, weight, dz, dweight, tokens, topk, rows, width,
                                                 stream));
}

}  // extern "C"
