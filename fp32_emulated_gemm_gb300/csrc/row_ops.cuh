// row_ops.cuh -- loads, stores and sums shared by the row-wise FP32 kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace emu {

inline bool vec4_ok(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld & 3) == 0; }

// (Plain loads: a kernel may write the matrix it reads, element by element.)
// Four values of a row: VEC: columns c .. c + 3 (all inside or all outside the
// row, whose width is a multiple of 4); otherwise columns c, c + S, c + 2S,
// c + 3S, each checked, so that neighbouring lanes read neighbouring words at
// any alignment.
template <bool VEC, int S>
__device__ __forceinline__ float4 load4(const float* row, int64_t c, int64_t n) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (VEC) {
        if (c < n) v = *reinterpret_cast<const float4*>(row + c);
    } else {
        if (c < n) v.x = row[c];
        if (c + S < n) v.y = row[c + S];
        if (c + 2 * S < n) v.z = row[c + 2 * S];
        if (c + 3 * S < n) v.w = row[c + 3 * S];
    }
    return v;
}
template <bool VEC, int S>
__device__ __forceinline__ void store4(float* row, int64_t c, int64_t n, const float4& v) {
    if constexpr (VEC) {
        if (c < n) *reinterpret_cast<float4*>(row + c) = v;
    } else {
        if (c < n) row[c] = v.x;
        if (c + S < n) row[c + S] = v.y;
        if (c + 2 * S < n) row[c + 2 * S] = v.z;
        if (c + 3 * S < n) row[c + 3 * S] = v.w;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sums over the rows of P x C partial sums: out0[c] for columns below `split`,
// out1[c - split] for the others (a null output is skipped).
struct Partials {
    const float* p;
    int P;
    int64_t C, split;
    float *out0, *out1;
};
// Up to two sets in one launch, as the dependent of the kernel launched on
// `stream` just before, which has to be this library's.
cudaError_t launch_sum_partials(const Partials* sets, int n, cudaStream_t stream);

}  // namespace emu
