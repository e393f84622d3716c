// Launches of any number of workgroups. Of a launch of 2^32 threads and more in
// one direction only their number modulo 2^32 runs, and the launch reports no
// error; so workgroups beyond 2^22 (2^32 threads are 2^23 of 512) go on in y:
// workgroup w is x = w % 2^22, y = w / 2^22. The last y may hold more
// workgroups than were asked for; a kernel ends those by its bounds. 2^22 is a
// multiple of the 8 XCDs, so w % 8 still names a workgroup's XCD.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libgemm {

constexpr int kWideBits = 22;
constexpr int64_t kMostWorkgroups = 0x7FFFFFFF - (1 << kWideBits);   // for kernels that count them in an int

// Whether x alone holds them (kernels that take no wide grid).
inline bool launch_holds(int64_t workgroups, int threads) { return workgroups <= 0xFFFFFFFFll / threads; }

inline dim3 wide_grid(int64_t workgroups) {
    const int64_t x = (int64_t)1 << kWideBits;
    return workgroups <= x ? dim3((unsigned)workgroups) : dim3((unsigned)x, (unsigned)((workgroups + x - 1) / x));
}

__device__ __forceinline__ int64_t wide_block() { return ((int64_t)blockIdx.y << kWideBits) + blockIdx.x; }

// Whether this workgroup is past the `count` asked for. Those of y = 0 never
// are, and need not wait for the count (4 x 11664 x 1040 with adapters: 13.88 us
// with the wait, 13.84 without).
__device__ __forceinline__ bool past_last_block(int64_t count) { return blockIdx.y != 0 && wide_block() >= count; }

}  // namespace libgemm
