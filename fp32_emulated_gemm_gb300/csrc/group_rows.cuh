// group_rows.cuh -- where the rows of a group lie, from the groups' offsets on the
// device, for the kernels of a few rows.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace emu {
namespace {

// The `at`-th of the blocks of MR rows at most that the groups' rows make, group by
// group, without the first SKIP of each: {first row, rows (0: there are fewer blocks),
// group}.  Each warp finds it for itself, 32 groups at a time: about 0.3 us, where a
// kernel of its own for a list of the blocks took 3.
template <int SKIP = 0>
__device__ __forceinline__ int3 rows_of_block(const int32_t* offsets, int groups, int M, int MR, int at) {
    const int lane = threadIdx.x & 31;
    int last = min(max(__ldcg(offsets), 0), M);  // where the groups so far end
    for (int base = 0; base < groups; base += 32) {
        // ends, made ascending
        int end = base + lane < groups ? min(max(__ldcg(offsets + base + lane + 1), 0), M) : 0;
        end = max(end, last);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, end, o);
            if (lane >= o) end = max(end, up);
        }
        const int prev = __shfl_up_sync(0xFFFFFFFFu, end, 1), first = lane == 0 ? last : prev;
        const int n = max((end - first + MR - 1) / MR - SKIP, 0);
        int through = n;  // blocks of this group and those before it
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, through, o);
            if (lane >= o) through += up;
        }
        const unsigned mine = __ballot_sync(0xFFFFFFFFu, at < through);
        if (mine) {
            const int src = __ffs(mine) - 1;
            const int f = __shfl_sync(0xFFFFFFFFu, first, src), e = __shfl_sync(0xFFFFFFFFu, end, src);
            const int b = at - __shfl_sync(0xFFFFFFFFu, through - n, src) + SKIP;
            return make_int3(f + b * MR, min(MR, e - f - b * MR), base + src);
        }
        at -= __shfl_sync(0xFFFFFFFFu, through, 31);
        last = __shfl_sync(0xFFFFFFFFu, end, 31);
    }
    return make_int3(0, 0, 0);
}

// Whether a group may have more than n rows; the whole block asks.  (No group of
// ascending offsets has more rows than its own two, clipped, are apart.)
__device__ __forceinline__ bool any_group_above(const int32_t* offsets, int groups, int M, int n) {
    bool above = false;
    for (int e = threadIdx.x; e < groups; e += blockDim.x)
        above |= min(max(__ldcg(offsets + e + 1), 0), M) - min(max(__ldcg(offsets + e), 0), M) > n;
    return __syncthreads_or(above);
}

// The rows [x, y) of one group; the whole warp asks.
__device__ __forceinline__ int2 rows_of_group(const int32_t* offsets, int M, int group) {
    const int lane = threadIdx.x & 31;
    int first = 0;  // the largest of the ends up to the group, made ascending and within the rows
    for (int e = lane; e <= group; e += 32) first = max(first, min(max(__ldcg(offsets + e), 0), M));
    first = __reduce_max_sync(0xFFFFFFFFu, first);
    return make_int2(first, max(first, min(max(__ldcg(offsets + group + 1), 0), M)));
}

}  // namespace
}  // namespace emu
