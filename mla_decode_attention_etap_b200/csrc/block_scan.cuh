// Block-wide prefix sum and minimum, used by the plan and by the kernels that keep the cache.
#pragma once

#include <cstdint>

namespace mla {

// Exclusive prefix sum of one int64 per thread over the block; *total gets the block sum.
__device__ __forceinline__ int64_t block_exclusive_scan(int64_t x, int64_t *smem32, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    int64_t incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) smem32[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int64_t w = lane < nwarps ? smem32[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += y;
        }
        smem32[lane] = w;  // inclusive prefix of the warp sums
    }
    __syncthreads();
    const int64_t base = warp > 0 ? smem32[warp - 1] : 0;
    *total = smem32[nwarps - 1];
    __syncthreads();  // smem32 is free for the next scan
    return base + incl - x;
}

// Minimum of one int per thread over the block (all threads call it).
__device__ __forceinline__ int block_min(int x, int *smem32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x = min(x, __shfl_xor_sync(0xffffffffu, x, d));
    if (lane == 0) smem32[warp] = x;
    __syncthreads();
    int r = smem32[0];
    for (int w = 1; w < nwarps; ++w) r = min(r, smem32[w]);
    __syncthreads();
    return r;
}

}  // namespace mla
