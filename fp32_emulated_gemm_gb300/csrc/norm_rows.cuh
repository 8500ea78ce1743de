// norm_rows.cuh -- what the norms over rows (layer_norm.cu, rms_norm.cu) share:
// threads that share a row, their sums, and how many blocks a launch takes.
#pragma once

#include <cuda_runtime.h>

#include "row_ops.cuh"

namespace emu {
namespace {

// ------------------------------------------------- rows held in registers --
// T threads share a row and hold it in NV float4 each (4 T NV >= N), so X and
// dY are read once.  T <= 32: part of a warp or a warp a row, sums by shuffles
// alone.  Wider rows take a block each, whose sums cost barriers: there few
// threads with many values each keep the most rows in flight per SM.
template <int T> constexpr int kBlockThreads = T <= 32 ? 256 : T;
template <int T> constexpr int kBlockRows = T <= 32 ? 256 / T : 1;

// Sums over the T threads of a row of two values, returned to all of them.
// `flip` alternates between two sets of slots from one call to the next, so
// one barrier per call is enough.
template <int T>
__device__ __forceinline__ float2 row_sum2(float a, float b, int& flip) {
#pragma unroll
    for (int o = T < 32 ? T / 2 : 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if constexpr (T <= 32) return make_float2(a, b);
    __shared__ float2 part[2][T / 32 + 1];
    float2* p = part[flip];
    flip ^= 1;
    if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 s = p[0];
#pragma unroll
    for (int i = 1; i < T / 32; ++i) { s.x += p[i].x; s.y += p[i].y; }
    return s;
}

// Column of value j of float4 i of thread t (see load4).
template <int T, bool VEC> __device__ __forceinline__ int64_t col_of(int t, int i) {
    return (VEC ? 4 * t : t) + (int64_t)4 * T * i;
}
template <int T, bool VEC> __device__ __forceinline__ bool inside(int64_t c, int j, int64_t n) {
    return VEC ? c < n : c + j * T < n;
}

// Blocks of a kernel that are resident on an SM at once (asked for once; the
// library holds code for one architecture).
template <class K> int resident_blocks(K kernel, int threads) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = 1;
    }
    return n;
}

// Blocks that take the rows in turns of equal length: at most `resident`.
unsigned even_grid(int64_t M, int rows, int64_t resident) {
    const int64_t groups = (M + rows - 1) / rows, turns = (groups + resident - 1) / resident;
    return (unsigned)((groups + turns - 1) / turns);
}

// Rows wider than the registers hold: a block a row.
constexpr int kRowThreads = 256;

// Sum over the block of two values, returned to every thread.
__device__ __forceinline__ float2 block_sum2(float a, float b) {
    __shared__ float2 part[kRowThreads / 32];
    a = warp_sum(a);
    b = warp_sum(b);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
    for (int i = 0; i < kRowThreads / 32; ++i) { s.x += part[i].x; s.y += part[i].y; }
    return s;
}

}  // namespace
}  // namespace emu
