// Internal interface between the C-ABI layer, the shape selector and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libgemm {

enum OperandKind { KIND_F16 = 0, KIND_FP8 = 1 };

// Arguments every GEMM launcher receives (validated by the C-ABI layer).
struct GemmArgs {
    const void* A;
    const void* B;
    void* C;
    const float* sA;   // device scalars (per-channel: sA[M], sB[N]); NULL for FP16
    const float* sB;
    const float* sOut; // device scalar; only read for FP8 outputs
    int out_dtype;
    int64_t M, N, K;
    hipStream_t stream;
    int fmt_a = 0;     // FP8 operand formats (Fp8Format: 0 = E4M3, 1 = E5M2); 0 for FP16
    int fmt_b = 0;
    int channel = 0;   // 1: sA holds M per-row scales and sB N per-column scales
    // Split-K: with splits > 1 the launch covers K in ranges of k_chunk and
    // writes FP32 partial sums to ws[split][M][N] instead of C; the reduce
    // launch (launch_splitk_reduce) then writes C.
    float* ws = nullptr;
    int splits = 1;
    int64_t k_chunk = 0;
    // 1: B is stored K-major, as Bt[N,K] row-major (element (k, n) at n*K + k)
    int b_kmajor = 0;
};

// Products whose weight depends on the row: the arguments of a plain product
// with M = rows, and the cut of the rows into groups (row_groups.h).
struct GroupedArgs : GemmArgs {
    const int32_t* offsets = nullptr;   // device, groups + 1
    int64_t groups = 0;
};

// A product with K-major weight plus the low-rank term of each row's adapter.
struct LoraArgs : GemmArgs {
    const void* X = nullptr;            // FP16 [M, K]: what the adapters multiply (A itself for FP16)
    const void* LA = nullptr;           // FP16 [adapters, rank, K]
    const void* LB = nullptr;           // FP16 [adapters, N, rank]
    const int32_t* adapter = nullptr;   // device, M: the row's adapter, none outside [0, adapters)
    const float* lscale = nullptr;      // device, adapters
    int64_t rank = 0, adapters = 0;
    float* low = nullptr;               // workspace: slices of [M, rank rounded up to 8]
    int low_slices = 1;                 // parts of the low-rank values, which the products add up
};

// A product with bias, activation and residual in its epilogue.
struct BiasActArgs : GemmArgs {
    const float* bias = nullptr;        // device, N; or NULL
    const void* residual = nullptr;     // device, [M, N] of res_dtype; or NULL
    void* Z = nullptr;                  // device, [M, N] of z_dtype: the values before the activation; or NULL
    uint8_t* zscale = nullptr;          // their scales, 8-bit values (row_io.h)
    int act = 0;                        // Activation (act.h)
    int res_dtype = 0, z_dtype = 0;     // OutDtype
};

typedef hipError_t (*GemmLauncher)(const GemmArgs&);

// One entry of the compiled-in configuration table.
struct GemmConfig {
    const char* name;   // e.g. "tile_fp8_256x256x128_w2x2"
    int kind;           // OperandKind
    int family;         // 0 = MFMA tile kernel, 1 = M<=16 streaming kernel, 2 = direct-load tile kernel,
                        // 3 = K-major decode kernel, 4 = ping-pong tile kernel,
                        // 5 = exact-accumulation FP8 tile kernel, 6 = deep-ring skinny kernel
    int bm, bn, bk;     // tile (stream: bm = max M, bn = columns per block, bk = k-slices)
    GemmLauncher launch;
    int fmt_mask = 0;   // FP8 operand pairs served: bit (2*fmt_a + fmt_b); 0 means E4M3 x E4M3 only
    int kgran = 0;      // split-K: K ranges are multiples of kgran; 0 = this config does not split
    int b_kmajor = 0;   // B layout served: 0 row-major B[K,N], 1 K-major Bt[N,K]
};

constexpr int kAllFp8Pairs = 15;

// Whether configuration c serves FP8 operand formats (fa, fb).
inline bool serves_formats(const GemmConfig& c, int fa, int fb) {
    const int mask = c.fmt_mask ? c.fmt_mask : 1;
    return (mask >> (2 * fa + fb)) & 1;
}

// Configuration tables, defined next to their kernels.
const GemmConfig* tile_configs(int* count);
const GemmConfig* stream_configs(int* count);
const GemmConfig* dma_configs(int* count);
const GemmConfig* gemv_kmajor_configs(int* count);
const GemmConfig* pp_configs(int* count);
const GemmConfig* exact_configs(int* count);
// exact-accumulation ping-pong launchers (gemm_pp_exact.hip), row-major / K-major B
hipError_t launch_pp_exact_rm(const GemmArgs& a);
hipError_t launch_pp_exact_bt(const GemmArgs& a);
const GemmConfig* ring_configs(int* count);

// Shape (and FP8 operand formats) -> configuration (host only, no HIP calls).
// Returns NULL if none fits.
const GemmConfig* select_config(int kind, int out_dtype, int64_t M, int64_t N, int64_t K, int fmt_a = 0,
                                int fmt_b = 0, int b_kmajor = 0);

// Split-K plan for the workspace entry points: the configuration, the number
// of K ranges and their length (splits == 1: no split, the plain launch).
struct SplitPlan {
    const GemmConfig* cfg;
    int splits;
    int64_t k_chunk;
};
// The exact-accumulation FP8 mode: the FP32-FMA streaming (row-major B,
// M <= 4) and decode (K-major B, M <= 8) kernels, whose products are exact and
// whose sums are FP32 additions, else the widening tile kernels by the tile
// rules. NULL if none fits.
const GemmConfig* select_config_exact(int out_dtype, int64_t M, int64_t N, int64_t K, int fmt_a, int fmt_b,
                                      int b_kmajor);

SplitPlan plan_splitk(int kind, int out_dtype, int64_t M, int64_t N, int64_t K, int fmt_a = 0, int fmt_b = 0,
                      int b_kmajor = 0);

// Products grouped by rows (routed.cpp chooses the kernel), kind: OperandKind.
hipError_t launch_grouped(int kind, const GroupedArgs& a);
// The register-staged tile kernel over row groups: any sizes and alignment.
hipError_t launch_grouped_tile_f16(const GroupedArgs& a, int bm);
hipError_t launch_grouped_tile_fp8(const GroupedArgs& a, int bm);
// C[g] = A[rows of g]^T B[rows of g] for FP16 A[rows, M], B[rows, N]; C F32 or
// F16 [groups, M, N]. K holds the number of rows.
hipError_t launch_grouped_wgrad(const GroupedArgs& a);
// low[i, r] = lscale[a_i] <X[i], LA[a_i, r]>, zero for rows without an adapter
// and from rank on, in a.low_slices parts, each the sum over a slice of K.
hipError_t launch_lora_low(const LoraArgs& a);
// Slices that launch_lora_low can use: the most for these rows and rank (what
// the workspace holds), and those for a call.
int lora_most_slices(int64_t rows, int64_t rank);
int lora_low_slices(const LoraArgs& a);
hipError_t launch_lora(int kind, const LoraArgs& a);
// Names of the kernels that these calls launch (host only).
const char* grouped_kernel_name(int kind, const GroupedArgs& a);
const char* wgrad_kernel_name(const GroupedArgs& a);
// launch_grouped_wgrad with A (qs 1) or B (qs 2) held as 8-bit values of format fmt
// and their scales (row_io.h); a.offsets may be NULL: one group of all rows.
hipError_t launch_wgrad_mx(const GroupedArgs& a, const uint8_t* scale, int fmt, int qs);
const char* wgrad_mx_kernel_name(const GroupedArgs& a, int qs);
const char* lora_kernel_name(int kind, const LoraArgs& a);
hipError_t launch_lora_tile_f16(const LoraArgs& a, int bm);
hipError_t launch_lora_tile_fp8(const LoraArgs& a, int bm);
// The deep-ring kernel over row groups of few rows / with adapters, for
// operands it takes.
bool grouped_ring_takes_f16(const GroupedArgs& a);
bool grouped_ring_takes_fp8(const GroupedArgs& a);
hipError_t launch_grouped_ring_f16(const GroupedArgs& a);
hipError_t launch_grouped_ring_fp8(const GroupedArgs& a);
// The deep ring's tiles for adapters, and the one that the plain product's rule
// picks: the fewest bytes a compute unit streams (in 128-byte rows of A and B
// per K tile), ties to the larger tile.
constexpr int kLoraRingShapes[][2] = {{16, 16}, {16, 32}, {16, 64}, {32, 32}, {32, 64}, {64, 64}};
inline int lora_ring_shape(int64_t M, int64_t N, int64_t* cost) {
    int pick = -1, at = 0;
    for (const auto& c : kLoraRingShapes) {
        const int64_t tiles = ((M + c[0] - 1) / c[0]) * ((N + c[1] - 1) / c[1]);
        const int64_t bytes = ((tiles + 255) / 256) * (c[0] + c[1]);
        if (pick < 0 || bytes < *cost ||
            (bytes == *cost && c[0] * c[1] > kLoraRingShapes[pick][0] * kLoraRingShapes[pick][1])) {
            pick = at;
            *cost = bytes;
        }
        ++at;
    }
    return pick;
}
bool lora_ring_takes_f16(const LoraArgs& a);
bool lora_ring_takes_fp8(const LoraArgs& a);
hipError_t launch_lora_ring_f16(const LoraArgs& a);
hipError_t launch_lora_ring_fp8(const LoraArgs& a);
// The ping-pong tile kernel over row groups / with adapters: whether it takes
// the operands (16-byte alignment, 32-bit offsets), and its launches (bm 128, 192
// or 256 rows, adapters 192 or 256; pairs with E5M2: 192).
bool grouped_pp_takes_f16(const GroupedArgs& a);
bool grouped_pp_takes_fp8(const GroupedArgs& a);
bool lora_pp_takes_f16(const LoraArgs& a);
bool lora_pp_takes_fp8(const LoraArgs& a);
hipError_t launch_grouped_pp_f16(const GroupedArgs& a, int bm);
hipError_t launch_grouped_pp_e4m3(const GroupedArgs& a, int bm);
hipError_t launch_grouped_pp_mixed(const GroupedArgs& a);
hipError_t launch_lora_pp_f16(const LoraArgs& a, int bm);
hipError_t launch_lora_pp_e4m3(const LoraArgs& a, int bm);
hipError_t launch_lora_pp_mixed(const LoraArgs& a);

// Products with bias, activation and residual (bias_act.cpp chooses the kernel).
hipError_t launch_bias_act(int kind, const BiasActArgs& a);
const char* bias_act_kernel_name(int kind, const BiasActArgs& a);
hipError_t launch_bias_act_gemv_f16(const BiasActArgs& a);
bool bias_act_ring_takes(int kind, const BiasActArgs& a);
hipError_t launch_bias_act_ring_f16(const BiasActArgs& a, int shape);
hipError_t launch_bias_act_ring_fp8(const BiasActArgs& a, int shape);   // shape: of kLoraRingShapes
bool bias_act_pp_takes_f16(const BiasActArgs& a);
bool bias_act_pp_takes_fp8(const BiasActArgs& a);
hipError_t launch_bias_act_pp_f16(const BiasActArgs& a, int bm);
hipError_t launch_bias_act_pp_e4m3(const BiasActArgs& a, int bm);
hipError_t launch_bias_act_pp_mixed(const BiasActArgs& a);
hipError_t launch_bias_act_tile_f16(const BiasActArgs& a, int bm);
hipError_t launch_bias_act_tile_fp8(const BiasActArgs& a, int bm);

// C = epilogue(sum over a.splits slices of a.ws), in slice order.
hipError_t launch_splitk_reduce(const GemmArgs& a);

// amax / quantize launchers.
// amax and (scale != NULL) the scale for FP8 format fmt, pow2 != 0 for a
// power-of-two scale.
hipError_t launch_amax(const float* x, int64_t n, float* amax, float* scale, int fmt, int pow2, hipStream_t stream);
hipError_t launch_quantize(const float* x, int64_t n, const float* scale, uint8_t* q, int fmt, hipStream_t stream);
// amax, scale and quantize of two tensors in two launches (A, and B when
// nb > 0): amax[0..1], scale[0..1], qa, qb. slots: kPairSlots words of device
// scratch for the per-block maxima.
constexpr int kPairSlots = 1024;
hipError_t launch_amax_quantize_pair(const float* xa, int64_t na, const float* xb, int64_t nb, int fmt, int pow2,
                                     float* amax, float* scale, uint8_t* qa, uint8_t* qb, uint32_t* slots,
                                     hipStream_t stream);
// The same with B = xb[K, N] row-major and its codes written K-major, qbt[N, K].
hipError_t launch_amax_quantize_pair_bt(const float* xa, int64_t na, const float* xb, int64_t K, int64_t N, int fmt,
                                        int pow2, float* amax, float* scale, uint8_t* qa, uint8_t* qbt,
                                        uint32_t* slots, hipStream_t stream);
// Quantize with a transposed output: q[c * rows + r] = code(x[r * cols + c] / scale).
hipError_t launch_quantize_transposed(const float* x, int64_t rows, int64_t cols, const float* scale, uint8_t* q,
                                      int fmt, hipStream_t stream);
// Per-channel amax / scale / quantize over a row-major x[rows, cols]: axis 0
// one channel per row, axis 1 one per column. For axis 1, amax doubles as the
// running maximum while the launches run.
hipError_t launch_amax_channel(const float* x, int64_t rows, int64_t cols, int axis, float* amax, float* scale,
                               int fmt, int pow2, hipStream_t stream);
hipError_t launch_quantize_channel(const float* x, int64_t rows, int64_t cols, int axis, const float* scale,
                                   uint8_t* q, int fmt, hipStream_t stream);
// FP16 dynamic-range guard: scalars[0..2] = s, sqrt(s), 1/s from the two
// maxima (scale_out, if not NULL, receives s); y = FP16(fl32(x * sqrt(s))).
hipError_t launch_guard_scale(const float* amax_a, const float* amax_b, float* scalars, float* scale_out,
                              hipStream_t stream);
hipError_t launch_guard_to_f16(const float* x, int64_t n, const float* scalars, _Float16* y, hipStream_t stream);
// dst[c * rows + r] = src[r * cols + c] for 1- or 2-byte elements.
hipError_t launch_transpose(const void* src, int64_t rows, int64_t cols, int elem_bytes, void* dst,
                            hipStream_t stream);
// Writes zeros to an [M,N] output of the given dtype (the K = 0 empty sum).
hipError_t launch_fill_zero(void* C, int64_t count, int out_dtype, hipStream_t stream);

}  // namespace libgemm
