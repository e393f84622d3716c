// Internal interface of the norm, of the epilogue's gradient and of 8-bit values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libgemm {

// A compile-time number passed as a value (for generic lambdas).
template <int N>
struct IntC {
    static constexpr int value = N;
};

struct NormArgs {
    const void* x;          // [rows, width]
    const void* residual;   // or NULL
    const float* weight;    // [width]
    void* h;                // or NULL
    void* y;
    float* scale;           // [rows], FP8 outputs
    float* rstd;            // [rows] or NULL
    int64_t rows, width;
    float eps, inv_width;
    int pow2;
};

struct NormBackwardArgs {
    const void* dy;
    const void* h;
    const uint8_t* hscale;
    const float* weight;
    const float* rstd;
    const void* dh;         // or NULL
    void* dx;
    float* partial;         // workspace
    int64_t rows, width;
    float inv_width;
};

hipError_t launch_rms_norm(const NormArgs& a, int dtype, int out_dtype, hipStream_t s);
hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, int dtype, int h_dtype, float* dweight, hipStream_t s);
// Rows of partial sums of the gradient to the weights, and all FP32 words of the
// workspace (without that gradient: the long rows' own).
int64_t norm_backward_parts(int64_t rows, int64_t width);
int64_t norm_backward_words(int64_t rows, int64_t width, bool dweight);

// dz = dy act'(z), dbias = column sums of dz (FP32, before rounding).
struct ActBackwardArgs {
    const void* dy;
    const void* z;
    const uint8_t* zscale;
    void* dz;               // or NULL
    float* partial;         // workspace, or NULL without dbias
    int64_t rows, cols;
};

hipError_t launch_act_backward(const ActBackwardArgs& a, int dtype, int z_dtype, int act, float* dbias, hipStream_t s);
int64_t act_backward_parts(int64_t rows, int64_t cols);

// out[c] = sum over p < parts of partial[p, c], in a fixed order.
hipError_t launch_sum_parts(const float* partial, int64_t parts, int64_t cols, float* out, hipStream_t s);

hipError_t launch_quantize_mx(const void* x, int dtype, int64_t rows, int64_t cols, int fmt, uint8_t* q,
                              uint8_t* scale, hipStream_t s);
hipError_t launch_dequantize_mx(const uint8_t* q, const uint8_t* scale, int fmt, int64_t rows, int64_t cols, void* y,
                                int dtype, hipStream_t s);

}  // namespace libgemm
