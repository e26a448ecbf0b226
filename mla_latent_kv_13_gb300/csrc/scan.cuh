// scan.cuh -- prefix sums over a CTA.
#pragma once

#include <cuda_runtime.h>

namespace mla {

// Exclusive prefix sum of one value per thread over the CTA; *total (optional) the sum.
__device__ __forceinline__ int scan_block(int x, int *warp_tot, int *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_tot[w] = inc;
    __syncthreads();
    if (w == 0) {
        const int v = lane < static_cast<int>(blockDim.x >> 5) ? warp_tot[lane] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_tot[lane] = s - v;
        if (lane == 31) warp_tot[32] = s;
    }
    __syncthreads();
    const int before = warp_tot[w] + inc - x;
    *total = warp_tot[32];
    __syncthreads();
    return before;
}

}  // namespace mla
