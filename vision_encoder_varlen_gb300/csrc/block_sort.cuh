// Scan and sort of one 1024-thread block, and of one warp, shared by the work schedulers.
#pragma once

#include <stdint.h>

namespace vit {

constexpr int kSortThreads = 1024;

__device__ __forceinline__ int64_t block_exclusive_scan(int64_t v, int64_t *s_warp, int64_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;                // inclusive over warps
    }
    __syncthreads();
    const int64_t before = (warp > 0 ? s_warp[warp - 1] : 0) + x - v;
    *total = s_warp[31];
    __syncthreads();
    return before;
}

// Ascending bitonic sort of NPL (a power of two) keys in shared memory by the whole block.
__device__ __forceinline__ void block_sort(unsigned long long *s_key, int NPL, int tid)
{
    for (int k = 2; k <= NPL; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = tid; i < NPL; i += kSortThreads) {
                const int l = i ^ j;
                if (l > i) {
                    const unsigned long long x = s_key[i], y = s_key[l];
                    const bool up = (i & k) == 0;
                    if ((x > y) == up) {
                        s_key[i] = y;
                        s_key[l] = x;
                    }
                }
            }
            __syncthreads();
        }
    }
}

// For up to 32 keys, one per lane (all different): the lane's place in ascending order, and the sums of n0 and n1
// over the lanes placed before it.
__device__ __forceinline__ void warp_place(unsigned long long key, int n0, int n1, int &rank, int &at0, int &at1)
{
    rank = at0 = at1 = 0;
#pragma unroll 4
    for (int j = 0; j < 32; ++j) {
        const unsigned long long other = __shfl_sync(0xffffffffu, key, j);
        const int m0 = __shfl_sync(0xffffffffu, n0, j), m1 = __shfl_sync(0xffffffffu, n1, j);
        if (other < key) {
            ++rank;
            at0 += m0;
            at1 += m1;
        }
    }
}

// The last p < n with first(p) <= i, for items whose list is sorted by first = s_key >> 32.
__device__ __forceinline__ int place_of(const unsigned long long *s_key, int n, int i)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if ((int)(s_key[m] >> 32) <= i) lo = m;
        else hi = m;
    }
    return lo;
}

}  // namespace vit
