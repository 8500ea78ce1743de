// exchange.cu -- tokens to their experts' rows and back.
//
// A plan (route.cu) gives each of a token's k choices a row (slots[m, j], -1:
// none) and each row its choice (sources[row], -1: none).
//   dispatch     Xs[slots[m, j]] = X[m], rows without a source 0
//   combine      Y[m] = sum_j w[m, j] Ys[slots[m, j]] (+ R[m]); without weights
//                that is dispatch's gradient too
//   combine_bwd  dYs[slots[m, j]] = w[m, j] dY[m], rows without a source 0;
//                dw[m, j] = <dY[m], Ys[slots[m, j]]>
// Bound by memory.  All go through the tokens, T lanes each: a token's row is
// read once for its k copies, which are whole rows wherever they lie, and the
// sum over the choices is one thread's, in order: no atomics.
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"
#include "row_ops.cuh"

namespace emu {
namespace {

constexpr int kThreads = 256, kMaxChoices = 32;

struct Exchange {
    int64_t M, N, rows;  // rows: M k
    int k;
    const int32_t *slots, *sources;
    const float* weights;
    const float* A;      // dispatch: X; combine: Ys; combine_bwd: dY
    int64_t lda;
    const float* R;      // combine: residual; combine_bwd: Ys (for dw)
    int64_t ldr;
    float* C;            // dispatch: Xs; combine: Y; combine_bwd: dYs
    int64_t ldc;
    float* dweights;
};

__device__ __forceinline__ float4 scale4(const float4& v, float w) {
    return make_float4(v.x * w, v.y * w, v.z * w, v.w * w);
}

// (a slot outside the rows counts as none)
__device__ __forceinline__ int64_t slot_of(const Exchange& p, int64_t m, int j) {
    const int32_t s = __ldg(p.slots + m * p.k + j);
    return (uint32_t)s < (uint32_t)p.rows ? s : -1;
}

// Zeros in the rows that have no source.
template <int T, bool VEC> __device__ __forceinline__ void clear_rows(const Exchange& p) {
    const int t = threadIdx.x % T;
    const int64_t step = (int64_t)gridDim.x * (kThreads / T);
    for (int64_t r = blockIdx.x * (int64_t)(kThreads / T) + threadIdx.x / T; r < p.rows; r += step) {
        if (__ldg(p.sources + r) >= 0) continue;
        for (int64_t c = VEC ? 4 * t : t; c < p.N; c += 4 * T)
            store4<VEC, T>(p.C + r * p.ldc, c, p.N, make_float4(0.f, 0.f, 0.f, 0.f));
    }
}

// BWD: scaled by the weights, with their gradients.
template <int T, int NV, bool VEC, bool BWD>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const __grid_constant__ Exchange p) {
    const int t = threadIdx.x % T;
    const int64_t step = (int64_t)gridDim.x * (kThreads / T);
    for (int64_t base = blockIdx.x * (int64_t)(kThreads / T); base < p.M; base += step) {
        const int64_t m = base + threadIdx.x / T;
        const bool real = m < p.M;
        float mine[BWD ? kMaxChoices / T + (kMaxChoices % T != 0) : 1] = {};  // lane j % T's sum of choice j
        for (int64_t c0 = 0; c0 < p.N; c0 += 4 * T * NV) {
            float4 x[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i)
                x[i] = load4<VEC, T>(p.A + m * p.lda, c0 + (VEC ? 4 * t : t) + 4 * T * i, real ? p.N : 0);
            for (int j = 0; j < p.k; ++j) {
                const int64_t s = real ? slot_of(p, m, j) : -1;
                const int64_t n = s >= 0 ? p.N : 0;
                if constexpr (!BWD) {
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        store4<VEC, T>(p.C + s * p.ldc, c0 + (VEC ? 4 * t : t) + 4 * T * i, n, x[i]);
                } else {
                    const float w = s >= 0 ? __ldg(p.weights + m * p.k + j) : 0.f;
                    float dot = 0.f;
                    if (p.dweights) {
                        float4 y[NV];
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            y[i] = load4<VEC, T>(p.R + s * p.ldr, c0 + (VEC ? 4 * t : t) + 4 * T * i, n);
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            dot += fmaf(x[i].x, y[i].x, x[i].y * y[i].y) + fmaf(x[i].z, y[i].z, x[i].w * y[i].w);
                    }
                    if (p.C) {
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            store4<VEC, T>(p.C + s * p.ldc, c0 + (VEC ? 4 * t : t) + 4 * T * i, n, scale4(x[i], w));
                    }
                    if (p.dweights) {
#pragma unroll
                        for (int o = T / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
#pragma unroll
                        for (int q = 0; q < (int)(sizeof(mine) / sizeof(float)); ++q)
                            if (j == t + T * q) mine[q] += dot;
                    }
                }
            }
        }
        if constexpr (BWD) {
            if (p.dweights && real) {
#pragma unroll
                for (int q = 0; q < (int)(sizeof(mine) / sizeof(float)); ++q)
                    if (t + T * q < p.k) p.dweights[m * p.k + t + T * q] = mine[q];
            }
        }
    }
    if (p.C) clear_rows<T, VEC>(p);
}

template <int T, int NV, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ Exchange p) {
    const int t = threadIdx.x % T;
    const int64_t step = (int64_t)gridDim.x * (kThreads / T);
    for (int64_t m = blockIdx.x * (int64_t)(kThreads / T) + threadIdx.x / T; m < p.M; m += step) {
        for (int64_t c0 = 0; c0 < p.N; c0 += 4 * T * NV) {
            float4 s[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j = 0; j < p.k; ++j) {
                const int64_t r = slot_of(p, m, j);
                const int64_t n = r >= 0 ? p.N : 0;
                const float w = p.weights ? __ldg(p.weights + m * p.k + j) : 1.f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const float4 v = load4<VEC, T>(p.A + r * p.lda, c0 + (VEC ? 4 * t : t) + 4 * T * i, n);
                    if (r >= 0)
                        s[i] = make_float4(fmaf(w, v.x, s[i].x), fmaf(w, v.y, s[i].y), fmaf(w, v.z, s[i].z),
                                           fmaf(w, v.w, s[i].w));
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = c0 + (VEC ? 4 * t : t) + 4 * T * i;
                if (p.R) {
                    const float4 q = load4<VEC, T>(p.R + m * p.ldr, c, p.N);
                    s[i] = make_float4(s[i].x + q.x, s[i].y + q.y, s[i].z + q.z, s[i].w + q.w);
                }
                store4<VEC, T>(p.C + m * p.ldc, c, p.N, s[i]);
            }
        }
    }
}

template <class F> void for_width(int64_t N, F f) {
    auto of = [&](auto T, auto NV) { f(T, NV); };
    using std::integral_constant;
#define EMU_WIDTH(T, NV) of(integral_constant<int, T>{}, integral_constant<int, NV>{})
    if (N <= 16) EMU_WIDTH(4, 1);
    else if (N <= 32) EMU_WIDTH(8, 1);
    else if (N <= 64) EMU_WIDTH(16, 1);
    else if (N <= 128) EMU_WIDTH(32, 1);
    else if (N <= 256) EMU_WIDTH(32, 2);
    else EMU_WIDTH(32, 4);
#undef EMU_WIDTH
}

enum Kind { DISPATCH, COMBINE, COMBINE_BWD };

emu_status_t launch(Kind kind, const Exchange& p, emu_stream_t stream) {
    DeviceCtx dev;
    const emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = (p.N & 3) == 0 && vec4_ok(p.A, p.lda) && vec4_ok(p.R, p.R ? p.ldr : 0) && vec4_ok(p.C, p.C ? p.ldc : 0);
    cudaGetLastError();
    for_width(p.N, [&](auto T, auto NV) {
        constexpr int t = decltype(T)::value, nv = decltype(NV)::value;
        const int64_t groups = (p.M + kThreads / t - 1) / (kThreads / t), most = (int64_t)dev.sm_count * 8;
        const unsigned grid = (unsigned)(groups < most ? groups : most);
        auto go = [&](auto VEC) {
            constexpr bool v = decltype(VEC)::value;
            if (kind == DISPATCH) dispatch_kernel<t, nv, v, false><<<grid, kThreads, 0, s>>>(p);
            else if (kind == COMBINE) combine_kernel<t, nv, v><<<grid, kThreads, 0, s>>>(p);
            else dispatch_kernel<t, nv, v, true><<<grid, kThreads, 0, s>>>(p);
        };
        if (vec) go(std::true_type{}); else go(std::false_type{});
    });
    return cudaGetLastError() == cudaSuccess ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED;
}

emu_status_t sizes(int64_t M, int k, int64_t N) {
    if (M < 0 || k < 1 || N < 0) return EMU_STATUS_INVALID_VALUE;
    if (k > kMaxChoices || M > (INT32_MAX - 256) / k || N > INT32_MAX - 256) return EMU_STATUS_NOT_SUPPORTED;
    return EMU_STATUS_SUCCESS;
}

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" {

emu_status_t emu_expert_dispatch(int64_t M, int k, int64_t N, const float* X, int64_t ldx, const int32_t* slots,
                                 const int32_t* sources, float* Xs, int64_t ldxs, emu_stream_t stream) {
    const emu_status_t st = sizes(M, k, N);
    if (st != EMU_STATUS_SUCCESS || M == 0 || N == 0) return st;
    if (!X || !slots || !sources || !Xs || ldx < N || ldxs < N) return EMU_STATUS_INVALID_VALUE;
    return launch(DISPATCH, {M, N, M * k, k, slots, sources, nullptr, X, ldx, nullptr, 0, Xs, ldxs, nullptr}, stream);
}

emu_status_t emu_expert_combine_fwd(int64_t M, int k, int64_t N, const float* Ys, int64_t ldys, const int32_t* slots,
                                    const float* weights, const float* residual, int64_t ldr, float* Y, int64_t ldy,
                                    emu_stream_t stream) {
    const emu_status_t st = sizes(M, k, N);
    if (st != EMU_STATUS_SUCCESS || M == 0 || N == 0) return st;
    if (!Ys || !slots || !Y || ldys < N || ldy < N || (residual && ldr < N)) return EMU_STATUS_INVALID_VALUE;
    return launch(COMBINE, {M, N, M * k, k, slots, nullptr, weights, Ys, ldys, residual, ldr, Y, ldy, nullptr}, stream);
}

emu_status_t emu_expert_combine_bwd(int64_t M, int k, int64_t N, const float* dY, int64_t lddy, const float* Ys,
                                    int64_t ldys, const int32_t* slots, const int32_t* sources, const float* weights,
                                    float* dYs, int64_t lddys, float* dweights, emu_stream_t stream) {
    const emu_status_t st = sizes(M, k, N);
    if (st != EMU_STATUS_SUCCESS || M == 0) return st;
    if (!slots || (N > 0 && (!dY || lddy < N)) || (dYs && (!sources || !weights || lddys < N)) ||
        (dweights && N > 0 && (!Ys || ldys < N)))
        return EMU_STATUS_INVALID_VALUE;
    if (!dYs && !dweights) return EMU_STATUS_SUCCESS;
    if (N == 0) {  // empty products
        if (!dweights) return EMU_STATUS_SUCCESS;
        DeviceCtx dev;
        const emu_status_t ds = current_device(&dev);
        if (ds != EMU_STATUS_SUCCESS) return ds;
        if (cudaMemsetAsync(dweights, 0, (size_t)M * k * sizeof(float), reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();
            return EMU_STATUS_LAUNCH_FAILED;
        }
        return EMU_STATUS_SUCCESS;
    }
    return launch(COMBINE_BWD, {M, N, M * k, k, slots, sources, weights, dY, lddy, dweights ? Ys : nullptr, ldys, dYs, lddys,
                                dweights}, stream);
}

}  // extern "C"
