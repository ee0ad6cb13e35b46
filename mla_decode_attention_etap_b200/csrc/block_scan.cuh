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

// The same for two values at once (smem64: 64 words).
__device__ __forceinline__ void block_exclusive_scan2(int64_t &x, int64_t &y, int64_t *smem64, int64_t *total_x,
                                                      int64_t *total_y) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    int64_t ix = x, iy = y;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, ix, d), b = __shfl_up_sync(0xffffffffu, iy, d);
        if (lane >= d) {
            ix += a;
            iy += b;
        }
    }
    if (lane == 31) {
        smem64[warp] = ix;
        smem64[32 + warp] = iy;
    }
    __syncthreads();
    if (warp < 2) {  // one warp per value
        int64_t w = lane < nwarps ? smem64[32 * warp + lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += a;
        }
        smem64[32 * warp + lane] = w;  // inclusive prefix of the warp sums
    }
    __syncthreads();
    x = (warp > 0 ? smem64[warp - 1] : 0) + ix - x;
    y = (warp > 0 ? smem64[32 + warp - 1] : 0) + iy - y;
    *total_x = smem64[nwarps - 1];
    *total_y = smem64[32 + nwarps - 1];
    __syncthreads();  // smem64 is free for the next scan
}

// Minimum of one int per thread over the block (all threads call it).
__device__ __forceinline__ int block_min(int x, int *smem32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    x = __reduce_min_sync(0xffffffffu, x);
    if (lane == 0) smem32[warp] = x;
    __syncthreads();
    const int r = __reduce_min_sync(0xffffffffu, lane < nwarps ? smem32[lane] : 0x7fffffff);
    __syncthreads();
    return r;
}

}  // namespace mla
