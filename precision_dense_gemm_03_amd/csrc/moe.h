// Internal interface of the expert-routing kernels (moe_route.hip, moe_rows.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libgemm {

constexpr int kRouteMaxExperts = 1024;  // 64 logits per lane in registers
constexpr int kRouteMaxTopk = 32;       // two choices per lane
constexpr int kRouteMaxBlocks = 256;    // workgroups whose counts the second launch adds

struct RouteArgs {
    const float* logits;   // [T, E]
    int64_t T, E, K;
    int renorm;
    int32_t* expert;       // [T, K]
    float* weight;         // [T, K]
    int32_t* offsets;      // [E + 1]
    int32_t* row;          // [T, K]
    int32_t* token;        // [T * K]
    int32_t* counts;       // workspace, route_blocks(T) * E words when that is more than one block
    hipStream_t stream;
};

// Workgroups of the routing launches (and 64-token chunks per workgroup).
int route_blocks(int64_t T, int* per_block = nullptr);
hipError_t launch_route(const RouteArgs& a);
hipError_t launch_route_backward(const float* logits, const int32_t* expert, const float* weight,
                                 const float* dweight, int64_t T, int64_t E, int64_t K, int renorm, float* dlogits,
                                 hipStream_t stream);

// y[r] = x[token[r]], zeros where token[r] is no row of x[tokens, row_bytes].
hipError_t launch_moe_gather(const void* x, const int32_t* token, void* y, int64_t tokens, int64_t rows,
                             int64_t row_bytes, hipStream_t stream);
// y[t] = sum_j weight[t, j] z[row[t, j]] (weight NULL: 1); z, y: OUT_F32 or OUT_F16.
hipError_t launch_moe_combine(const void* z, int z_dtype, const int32_t* row, const float* weight, void* y,
                              int y_dtype, int64_t T, int64_t K, int64_t rows, int64_t width, hipStream_t stream);
// dz[row[t, j]] = weight[t, j] dy[t], dw[t, j] = <z[row[t, j]], dy[t]>; dy, z and dz of one type.
hipError_t launch_moe_combine_backward(const void* dy, const void* z, int dtype, const int32_t* row,
                                       const float* weight, void* dz, float* dw, int64_t T, int64_t K, int64_t rows,
                                       int64_t width, hipStream_t stream);

}  // namespace libgemm
