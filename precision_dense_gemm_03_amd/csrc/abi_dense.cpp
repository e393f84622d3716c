// C-ABI entry points of what a dense layer does around its products: the norm,
// products with bias, activation and residual, their gradients, and 8-bit values
// with scales (include/libgemm.h). Arguments are validated before any HIP call, as
// in abi.cpp.
#include "abi_common.h"
#include "act.h"
#include "kernels.h"
#include "norm.h"

using namespace libgemm;

namespace {

bool float_ok(int t) { return t == GEMM_OUT_F32 || t == GEMM_OUT_F16; }
bool any_ok(int t) { return t >= GEMM_OUT_F32 && t <= GEMM_OUT_E5M2; }
bool act_ok(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }
int64_t scales_of(int64_t rows, int64_t cols) { return rows * ((cols + 31) / 32); }

int bias_act_common(int kind, const void* A, int fmt_a, const void* B, int fmt_b, const float* sA, const float* sB,
                    int channel, const float* sOut, const float* bias, const void* residual, int res_dtype, void* C,
                    int out_dtype, int act, void* Z, uint8_t* Zscale, int z_dtype, int64_t M, int64_t N, int64_t K,
                    int b_kmajor, hipStream_t stream) {
    const int64_t es = kind == KIND_F16 ? 2 : 1;
    if (out_dtype < GEMM_OUT_F32 || out_dtype > (kind == KIND_F16 ? GEMM_OUT_F16 : GEMM_OUT_E5M2)) return GEMM_ERR_DTYPE;
    if (!fmt_ok(fmt_a) || !fmt_ok(fmt_b) || !act_ok(act)) return GEMM_ERR_DTYPE;
    if ((residual && !float_ok(res_dtype)) || (Z && !any_ok(z_dtype))) return GEMM_ERR_DTYPE;
    const int64_t os = out_size(out_dtype), zs = Z ? out_size(z_dtype) : 0, rs = residual ? out_size(res_dtype) : 0;
    const bool mx = Z && fp8_out(z_dtype);
    if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return GEMM_ERR_DIM;
    if (!bytes_ok(M, K, es) || !bytes_ok(K, N, es) || !bytes_ok(M, N, 4)) return GEMM_ERR_DIM;
    if (M == 0 || N == 0) return GEMM_OK;
    if (!C || (K > 0 && (!A || !B))) return GEMM_ERR_NULL;
    if (kind == KIND_FP8 && (!sA || !sB)) return GEMM_ERR_NULL;
    if ((fp8_out(out_dtype) && !sOut) || (mx && !Zscale)) return GEMM_ERR_SCALE;
    const Range w[3] = {{C, M * N * os}, {Z, M * N * zs}, {mx ? Zscale : nullptr, scales_of(M, N)}};
    const bool fp8 = kind == KIND_FP8;
    const Range r[7] = {{A, M * K * es}, {B, K * N * es}, {sA, fp8 ? (channel ? 4 * M : 4) : 0},
                        {sB, fp8 ? (channel ? 4 * N : 4) : 0}, {sOut, fp8_out(out_dtype) ? 4 : 0}, {bias, 4 * N},
                        {residual, M * N * rs}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    BiasActArgs a;
    static_cast<GemmArgs&>(a) = GemmArgs{A, B, C, sA, sB, fp8_out(out_dtype) ? sOut : nullptr, out_dtype, M, N, K,
                                         stream, fmt_a, fmt_b, channel ? 1 : 0};
    a.b_kmajor = b_kmajor;
    a.bias = bias;
    a.residual = residual;
    a.res_dtype = res_dtype;
    a.act = act;
    a.Z = Z;
    a.zscale = Zscale;
    a.z_dtype = z_dtype;
    return status_of(launch_bias_act(kind, a));
}

}  // namespace

static_assert(GEMM_ACT_NONE == ACT_NONE && GEMM_ACT_RELU == ACT_RELU && GEMM_ACT_GELU == ACT_GELU &&
                  GEMM_ACT_GELU_TANH == ACT_GELU_TANH && GEMM_ACT_SILU == ACT_SILU,
              "the activations' numbers");

extern "C" {

int rms_norm(const void* x, const void* residual, int dtype, const float* weight, float eps, void* h, void* y,
             int y_dtype, float* scale, int pow2, float* rstd, int64_t rows, int64_t width, hipStream_t stream) {
    if (!float_ok(dtype) || !any_ok(y_dtype)) return GEMM_ERR_DTYPE;
    if (!dim_ok(rows) || !dim_ok(width) || !bytes_ok(rows, width, 4)) return GEMM_ERR_DIM;
    if (rows == 0 || width == 0) return GEMM_OK;
    if (!x || !weight || !y) return GEMM_ERR_NULL;
    if (fp8_out(y_dtype) && !scale) return GEMM_ERR_SCALE;
    const int64_t n = rows * width, xs = n * out_size(dtype);
    const Range w[4] = {{h, xs}, {y, n * out_size(y_dtype)}, {fp8_out(y_dtype) ? scale : nullptr, 4 * rows},
                        {rstd, 4 * rows}};
    const Range r[3] = {{x, xs}, {residual, xs}, {weight, 4 * width}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    const NormArgs a{x, residual, weight, h, y, scale, rstd, rows, width, eps, 1.0f / (float)width, pow2};
    return status_of(launch_rms_norm(a, dtype, y_dtype, stream));
}

int64_t rms_norm_backward_workspace_size(int64_t rows, int64_t width) {
    if (!dim_ok(rows) || !dim_ok(width) || !bytes_ok(rows, width, 4)) return GEMM_ERR_DIM;
    return 4 * norm_backward_words(rows, width, true);
}

int rms_norm_backward(const void* dy, const void* dh, int dtype, const void* h, const uint8_t* hscale, int h_dtype,
                      const float* weight, const float* rstd, void* dx, float* dweight, int64_t rows, int64_t width,
                      void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!float_ok(dtype) || !any_ok(h_dtype)) return GEMM_ERR_DTYPE;
    if (!dim_ok(rows) || !dim_ok(width) || !bytes_ok(rows, width, 4)) return GEMM_ERR_DIM;
    if (width == 0 || (rows == 0 && !dweight)) return GEMM_OK;
    if (rows > 0 && (!dy || !h || !weight || !rstd || !dx)) return GEMM_ERR_NULL;
    const bool mx = fp8_out(h_dtype);
    if (rows > 0 && mx && !hscale) return GEMM_ERR_SCALE;
    const int64_t need = 4 * norm_backward_words(rows, width, dweight != nullptr);
    if (need > 0 && !workspace) return GEMM_ERR_NULL;
    if (need > 0 && (workspace_bytes < need || ((uintptr_t)workspace & 15u) != 0)) return GEMM_ERR_WORKSPACE;
    const int64_t n = rows * width, bytes = n * out_size(dtype);
    const Range w[3] = {{dx, bytes}, {dweight, 4 * width}, {need > 0 ? workspace : nullptr, need}};
    const Range r[6] = {{dy, bytes}, {dh, bytes}, {h, n * out_size(h_dtype)},
                        {mx ? hscale : nullptr, scales_of(rows, width)}, {weight, 4 * width}, {rstd, 4 * rows}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    if (rows == 0) return status_of(launch_fill_zero(dweight, width, GEMM_OUT_F32, stream));
    const NormBackwardArgs a{dy, h, hscale, weight, rstd, dh, dx, (float*)workspace, rows, width, 1.0f / (float)width};
    return status_of(launch_rms_norm_backward(a, dtype, h_dtype, dweight, stream));
}

int gemm_f16_bias_act(const void* A, const void* B, const float* bias, const void* residual, int res_dtype, void* C,
                      int out_dtype, int act, void* Z, uint8_t* Zscale, int z_dtype, int64_t M, int64_t N, int64_t K,
                      hipStream_t stream) {
    return bias_act_common(KIND_F16, A, 0, B, 0, nullptr, nullptr, 0, nullptr, bias, residual, res_dtype, C, out_dtype,
                           act, Z, Zscale, z_dtype, M, N, K, 0, stream);
}

int gemm_f16_bias_act_bt(const void* A, const void* Bt, const float* bias, const void* residual, int res_dtype, void* C,
                         int out_dtype, int act, void* Z, uint8_t* Zscale, int z_dtype, int64_t M, int64_t N,
                         int64_t K, hipStream_t stream) {
    return bias_act_common(KIND_F16, A, 0, Bt, 0, nullptr, nullptr, 0, nullptr, bias, residual, res_dtype, C,
                           out_dtype, act, Z, Zscale, z_dtype, M, N, K, 1, stream);
}

int gemm_fp8_bias_act(const uint8_t* A, int fmt_a, const uint8_t* B, int fmt_b, const float* sA, const float* sB,
                      int channel, const float* sOut, const float* bias, const void* residual, int res_dtype, void* C,
                      int out_dtype, int act, void* Z, uint8_t* Zscale, int z_dtype, int64_t M, int64_t N, int64_t K,
                      hipStream_t stream) {
    return bias_act_common(KIND_FP8, A, fmt_a, B, fmt_b, sA, sB, channel, sOut, bias, residual, res_dtype, C, out_dtype,
                           act, Z, Zscale, z_dtype, M, N, K, 0, stream);
}

int gemm_fp8_bias_act_bt(const uint8_t* A, int fmt_a, const uint8_t* Bt, int fmt_b, const float* sA, const float* sB,
                         int channel, const float* sOut, const float* bias, const void* residual, int res_dtype,
                         void* C, int out_dtype, int act, void* Z, uint8_t* Zscale, int z_dtype, int64_t M, int64_t N,
                         int64_t K, hipStream_t stream) {
    return bias_act_common(KIND_FP8, A, fmt_a, Bt, fmt_b, sA, sB, channel, sOut, bias, residual, res_dtype, C,
                           out_dtype, act, Z, Zscale, z_dtype, M, N, K, 1, stream);
}

int gemm_select_config_bias_act(int kind, int out_dtype, int64_t M, int64_t N, int64_t K, int fmt_a, int fmt_b,
                                int b_kmajor, int z_dtype, char* buf, int buflen) {
    if (kind != KIND_F16 && kind != KIND_FP8) return GEMM_ERR_DTYPE;
    if (out_dtype < GEMM_OUT_F32 || out_dtype > (kind == KIND_F16 ? GEMM_OUT_F16 : GEMM_OUT_E5M2)) return GEMM_ERR_DTYPE;
    if (kind == KIND_FP8 && (!fmt_ok(fmt_a) || !fmt_ok(fmt_b))) return GEMM_ERR_DTYPE;
    if (z_dtype >= 0 && !any_ok(z_dtype)) return GEMM_ERR_DTYPE;
    if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return GEMM_ERR_DIM;
    BiasActArgs a;
    static_cast<GemmArgs&>(a) = GemmArgs{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, out_dtype, M, N, K,
                                         nullptr, kind == KIND_F16 ? 0 : fmt_a, kind == KIND_F16 ? 0 : fmt_b, 0};
    a.b_kmajor = b_kmajor ? 1 : 0;
    a.Z = z_dtype >= 0 ? &a : nullptr;   // (only looked at for being there)
    a.z_dtype = z_dtype;
    return put_name(bias_act_kernel_name(kind, a), buf, buflen);
}

int64_t bias_act_backward_workspace_size(int64_t rows, int64_t cols) {
    if (!dim_ok(rows) || !dim_ok(cols) || !bytes_ok(rows, cols, 4)) return GEMM_ERR_DIM;
    return rows == 0 || cols == 0 ? 0 : 4 * act_backward_parts(rows, cols) * cols;
}

int bias_act_backward(const void* dy, int dtype, const void* Z, const uint8_t* Zscale, int z_dtype, int act, void* dZ,
                      float* dbias, int64_t rows, int64_t cols, void* workspace, int64_t workspace_bytes,
                      hipStream_t stream) {
    const bool reads_z = act != GEMM_ACT_NONE;
    if (!float_ok(dtype) || !act_ok(act) || (reads_z && !any_ok(z_dtype))) return GEMM_ERR_DTYPE;
    if (!dim_ok(rows) || !dim_ok(cols) || !bytes_ok(rows, cols, 4)) return GEMM_ERR_DIM;
    if (cols == 0 || (rows == 0 && !dbias)) return GEMM_OK;
    if (rows > 0 && (!dy || (reads_z && !Z) || (!dZ && !dbias))) return GEMM_ERR_NULL;
    const bool mx = reads_z && fp8_out(z_dtype);
    if (rows > 0 && mx && !Zscale) return GEMM_ERR_SCALE;
    const int64_t need = dbias ? bias_act_backward_workspace_size(rows, cols) : 0;
    if (need > 0 && !workspace) return GEMM_ERR_NULL;
    if (need > 0 && (workspace_bytes < need || ((uintptr_t)workspace & 15u) != 0)) return GEMM_ERR_WORKSPACE;
    const int64_t n = rows * cols, bytes = n * out_size(dtype);
    const Range w[3] = {{dZ, bytes}, {dbias, 4 * cols}, {need > 0 ? workspace : nullptr, need}};
    const Range r[3] = {{dy, bytes}, {Z, reads_z ? n * out_size(z_dtype) : 0}, {mx ? Zscale : nullptr, scales_of(rows, cols)}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    if (rows == 0) return status_of(launch_fill_zero(dbias, cols, GEMM_OUT_F32, stream));
    const ActBackwardArgs a{dy, Z, Zscale, dZ, dbias ? (float*)workspace : nullptr, rows, cols};
    return status_of(launch_act_backward(a, dtype, reads_z ? z_dtype : GEMM_OUT_F32, act, dbias, stream));
}

int quantize_mx_fp8(const void* x, int dtype, int64_t rows, int64_t cols, int fmt, uint8_t* q, uint8_t* scale,
                    hipStream_t stream) {
    if (!float_ok(dtype) || !fmt_ok(fmt)) return GEMM_ERR_DTYPE;
    if (!dim_ok(rows) || !dim_ok(cols) || !bytes_ok(rows, cols, 4)) return GEMM_ERR_DIM;
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (!x || !q || !scale) return GEMM_ERR_NULL;
    const Range w[2] = {{q, rows * cols}, {scale, scales_of(rows, cols)}};
    const Range r[1] = {{x, rows * cols * out_size(dtype)}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    return status_of(launch_quantize_mx(x, dtype, rows, cols, fmt, q, scale, stream));
}

int dequantize_mx_fp8(const uint8_t* q, const uint8_t* scale, int fmt, int64_t rows, int64_t cols, void* y, int dtype,
                      hipStream_t stream) {
    if (!float_ok(dtype) || !fmt_ok(fmt)) return GEMM_ERR_DTYPE;
    if (!dim_ok(rows) || !dim_ok(cols) || !bytes_ok(rows, cols, 4)) return GEMM_ERR_DIM;
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (!y || !q || !scale) return GEMM_ERR_NULL;
    const Range w[1] = {{y, rows * cols * out_size(dtype)}};
    const Range r[2] = {{q, rows * cols}, {scale, scales_of(rows, cols)}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    return status_of(launch_dequantize_mx(q, scale, fmt, rows, cols, y, dtype, stream));
}

int gemm_mx_wgrad(const uint8_t* Q, const uint8_t* Qscale, int fmt, const void* B, const int32_t* offsets, void* C,
                  int out_dtype, int64_t rows, int64_t M, int64_t N, int64_t groups, int q_second, hipStream_t stream) {
    if (!float_ok(out_dtype) || !fmt_ok(fmt)) return GEMM_ERR_DTYPE;
    const int64_t os = out_size(out_dtype);
    if (!size_ok(rows) || !size_ok(M) || !size_ok(N) || groups < 0 || groups > kMaxRowGroups) return GEMM_ERR_DIM;
    if (!bytes_ok(rows, M, 1) || !bytes_ok(rows, N, 2) || !bytes3_ok(M, N, groups, os)) return GEMM_ERR_DIM;
    if (!offsets && groups > 1) return GEMM_ERR_NULL;
    if (M == 0 || N == 0 || groups == 0) return GEMM_OK;
    if (!C || (rows > 0 && (!Q || !B))) return GEMM_ERR_NULL;
    if (rows > 0 && !Qscale) return GEMM_ERR_SCALE;
    const Range w[1] = {{C, groups * M * N * os}};
    const Range r[4] = {{Q, rows * M}, {Qscale, scales_of(rows, M)}, {B, rows * N * 2},
                        {offsets, offsets ? 4 * (groups + 1) : 0}};
    if (aliased(w, r)) return GEMM_ERR_ALIAS;
    const int st = check_device();
    if (st != GEMM_OK) return st;
    if (rows == 0) return status_of(launch_fill_zero(C, groups * M * N, out_dtype, stream));
    GroupedArgs a;
    if (q_second) static_cast<GemmArgs&>(a) = GemmArgs{B, Q, C, nullptr, nullptr, nullptr, out_dtype, N, M, rows, stream};
    else static_cast<GemmArgs&>(a) = GemmArgs{Q, B, C, nullptr, nullptr, nullptr, out_dtype, M, N, rows, stream};
    a.offsets = offsets;
    a.groups = groups;
    return status_of(launch_wgrad_mx(a, Qscale, fmt, q_second ? 2 : 1));
}

int gemm_select_config_mx_wgrad(int out_dtype, int64_t rows, int64_t M, int64_t N, int64_t groups, int q_second,
                                char* buf, int buflen) {
    if (!float_ok(out_dtype)) return GEMM_ERR_DTYPE;
    if (!size_ok(rows) || !size_ok(M) || !size_ok(N) || groups < 0 || groups > kMaxRowGroups) return GEMM_ERR_DIM;
    GroupedArgs a;
    static_cast<GemmArgs&>(a) = GemmArgs{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, out_dtype,
                                         q_second ? N : M, q_second ? M : N, rows, nullptr};
    a.groups = groups;
    return put_name(wgrad_mx_kernel_name(a, q_second ? 2 : 1), buf, buflen);
}

}  // extern "C"
