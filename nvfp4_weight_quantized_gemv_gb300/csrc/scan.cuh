// scan.cuh -- sums over a CTA's threads and searches in them, for the kernels
// that plan a batch's work.  They run once in a small kernel, most of whose time
// goes to fetching instructions: loops stay loops.
#pragma once

namespace nvfp4 {

constexpr int kMost = 0x7FFFFFFF;

// a + b for a, b in [0, kMost], kMost if it is more.
__device__ __forceinline__ int add_most(int a, int b) { return (int)min((unsigned)a + (unsigned)b, (unsigned)kMost); }

// Exclusive sums of N numbers over the CTA's threads, in place, none above kMost; total[i] is all threads'.
template <int N>
__device__ __forceinline__ void block_sums(int (&x)[N], int (&total)[N], int (*warps)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, all = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        int incl = x[i];
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl = add_most(incl, v);
        }
        if (lane == 31) warps[i][warp] = incl;
        incl = __shfl_up_sync(0xffffffffu, incl, 1);
        x[i] = lane ? incl : 0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        int sum = lane < all ? warps[i][lane] : 0;  // every warp scans the warps' sums
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum = add_most(sum, v);
        }
        total[i] = __shfl_sync(0xffffffffu, sum, 31);
        const int before = __shfl_sync(0xffffffffu, sum, (warp + 31) & 31);
        if (warp) x[i] = add_most(x[i], before);
    }
    __syncthreads();
}

// Last i of [0, n) with at[i] <= x (at[0] <= x, not decreasing).
__device__ __forceinline__ int last_at(const int *at, int n, int x) {
    int lo = 0;
#pragma unroll 1
    while (n > 1) {
        const int half = n >> 1;
        if (at[lo + half] <= x) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

}  // namespace nvfp4
