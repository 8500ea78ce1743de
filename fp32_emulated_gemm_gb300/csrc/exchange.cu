// exchange.cu -- tokens to their experts' rows and back.
//
// A plan (route.cu) gives each of a token's k choices a row (slots[m, j], -1:
// none) and each row its choice (sources[row], -1: none).
//   dispatch     Xs[slots[m, j]] = X[m], rows without a source 0
//   combine      Y[m] = sum_j w[m, j] Ys[slots[m, j]] (+ R[m]); without weights
//                that is dispatch's gradient too
//   combine_bwd  dYs[slots[m, j]] = w[m, j] dY[m], rows without a source 0;
//                dw[m, j] = <dY[m], Ys[slots[m, j]]>
// Bound by memory.  All go through the tokens, T lanes each (a block for each of a
// few wide ones): a token's row is read once for its k copies, which are whole rows
// wherever they lie, and the sum over the choices is one thread's, in order: no
// atomics.
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"
#include "norm_rows.cuh"

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

// A token's slots, T lanes a token: lane j has choice j's, asked for a token ahead
// so that the rows' loads do not wait for it; choices beyond the lanes are read
// where they are used.  A slot outside the rows counts as none.
template <int T> struct Slots {
    const Exchange& p;
    int32_t mine, next;
    float weight, next_weight;

    __device__ __forceinline__ Slots(const Exchange& e, int64_t m) : p(e) { ask(m); }
    __device__ __forceinline__ void ask(int64_t m) {
        const int t = threadIdx.x % T;
        const bool there = m < p.M && t < p.k;
        next = there ? __ldg(p.slots + m * p.k + t) : -1;
        next_weight = there && p.weights ? __ldg(p.weights + m * p.k + t) : 1.f;
    }
    // To the token asked for, and ask for the next.
    __device__ __forceinline__ void advance(int64_t m) {
        mine = next;
        weight = next_weight;
        ask(m);
    }
    __device__ __forceinline__ int64_t slot(int64_t m, int j) const {
        int32_t s = __shfl_sync(0xFFFFFFFFu, mine, j % T, T);
        if (j >= T) s = m < p.M ? __ldg(p.slots + m * p.k + j) : -1;
        return (uint32_t)s < (uint32_t)p.rows ? s : -1;
    }
    __device__ __forceinline__ float of(int64_t m, int j) const {
        float w = __shfl_sync(0xFFFFFFFFu, weight, j % T, T);
        if (j >= T) w = m < p.M && p.weights ? __ldg(p.weights + m * p.k + j) : 1.f;
        return w;
    }
};

// Zeros in the rows that have no source: a warp looks at up to 32 rows at a time,
// fewer where that leaves every warp some (they lie together, behind the others).
template <bool VEC> __device__ __forceinline__ void clear_rows(const Exchange& p) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    int chunk = 32;
    while (chunk > 1 && 4 * chunk * warps > p.rows) chunk /= 2;
    for (int64_t base = (blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5)) * chunk; base < p.rows; base += warps * chunk) {
        unsigned none = __ballot_sync(0xFFFFFFFFu, lane < chunk && base + lane < p.rows && __ldg(p.sources + base + lane) < 0);
        for (; none; none &= none - 1) {
            float* row = p.C + (base + __ffs(none) - 1) * p.ldc;
            for (int64_t c = VEC ? 4 * lane : lane; c < p.N; c += 128)
                store4<VEC, 32>(row, c, p.N, make_float4(0.f, 0.f, 0.f, 0.f));
        }
    }
}

__device__ __forceinline__ float dot4(const float4& a, const float4& b) {
    return fmaf(a.x, b.x, a.y * b.y) + fmaf(a.z, b.z, a.w * b.w);
}

// S groups of T lanes share a token's columns.  BWD: scaled by the weights, with
// their gradients.
template <int T, int NV, int S, bool VEC, bool BWD>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const __grid_constant__ Exchange p) {
    constexpr int kMine = BWD ? (kMaxChoices + T - 1) / T : 1, kTokens = kThreads / T / S;
    static_assert(S == 1 || T == 32, "the shared sums: a warp's lanes have a choice each");
    const int t = threadIdx.x % T, share = threadIdx.x / T % S;
    const int64_t step = (int64_t)gridDim.x * kTokens, first = share * (4 * T * NV);
    int64_t m = blockIdx.x * (int64_t)kTokens + threadIdx.x / (T * S);
    Slots<T> slots(p, m);
    float4 x[NV], ahead[NV];  // the token's row, and its first columns of the next token's
    auto load = [&](int64_t row, int64_t c0, float4 (&v)[NV]) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = load4<VEC, T>(p.A + row * p.lda, c0 + (VEC ? 4 * t : t) + 4 * T * i, row < p.M ? p.N : 0);
    };
    load(m, first, ahead);
    // (the loop is the same for all threads of a block: shuffles and barriers)
    for (int64_t base = blockIdx.x * (int64_t)kTokens; base < p.M; base += step, m += step) {
        slots.advance(m + step);
        const bool real = m < p.M;
        float mine[kMine] = {};  // dw of the choices t, t + T, ...
        for (int64_t c0 = first; c0 < p.N; c0 += 4 * T * NV * S) {
            const int64_t at = c0 + (VEC ? 4 * t : t);
            if (c0 == first) {
#pragma unroll
                for (int i = 0; i < NV; ++i) x[i] = ahead[i];
                load(m + step, first, ahead);
            } else {
                load(m, c0, x);
            }
            for (int j = 0; j < p.k; j += 2) {  // two choices' rows at a time
                int64_t s[2], n[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    s[q] = j + q < p.k ? slots.slot(m, j + q) : -1;
                    n[q] = s[q] >= 0 ? p.N : 0;
                }
                if constexpr (BWD) {
                    float4 y[2][NV];
                    if (p.dweights) {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int i = 0; i < NV; ++i) y[q][i] = load4<VEC, T>(p.R + s[q] * p.ldr, at + 4 * T * i, n[q]);
                    }
                    if (p.C) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float w = slots.of(m, j + q < p.k ? j + q : j);
#pragma unroll
                            for (int i = 0; i < NV; ++i)
                                store4<VEC, T>(p.C + s[q] * p.ldc, at + 4 * T * i, n[q], scale4(x[i], w));
                        }
                    }
                    if (p.dweights) {
                        float dot[2] = {0.f, 0.f};
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int i = 0; i < NV; ++i) dot[q] += dot4(x[i], y[q][i]);
#pragma unroll
                        for (int o = T / 2; o > 0; o >>= 1)
#pragma unroll
                            for (int q = 0; q < 2; ++q) dot[q] += __shfl_xor_sync(0xFFFFFFFFu, dot[q], o);
#pragma unroll
                        for (int i = 0; i < kMine; ++i)
#pragma unroll
                            for (int q = 0; q < 2; ++q)  // (none: 0, whatever is in dY)
                                if (j + q == t + T * i && s[q] >= 0) mine[i] += dot[q];
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < NV; ++i) store4<VEC, T>(p.C + s[q] * p.ldc, at + 4 * T * i, n[q], x[i]);
                }
            }
        }
        if constexpr (BWD) {
            if constexpr (S > 1) {
                if (p.dweights) {  // the shares' sums, added in order
                    __shared__ float sums[kTokens][S][T];
                    float* mine_of = sums[threadIdx.x / (T * S)][0];
                    mine_of[share * T + t] = mine[0];
                    __syncthreads();
#pragma unroll
                    for (int q = 1; q < S; ++q) mine[0] = q == 1 ? mine_of[t] + mine_of[T + t] : mine[0] + mine_of[q * T + t];
                    __syncthreads();
                }
            }
            if (p.dweights && real && share == 0) {
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (t + T * i < p.k) p.dweights[m * p.k + t + T * i] = mine[i];
            }
        }
    }
    if (p.C) clear_rows<VEC>(p);
}

template <int T, int NV, int S, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ Exchange p) {
    constexpr int kTokens = kThreads / T / S;
    const int t = threadIdx.x % T, share = threadIdx.x / T % S;
    const int64_t step = (int64_t)gridDim.x * kTokens;
    int64_t m = blockIdx.x * (int64_t)kTokens + threadIdx.x / (T * S);
    Slots<T> slots(p, m);
    for (int64_t base = blockIdx.x * (int64_t)kTokens; base < p.M; base += step, m += step) {
        slots.advance(m + step);
        const int64_t real = m < p.M ? p.N : 0;
        for (int64_t c0 = share * (4 * T * NV); c0 < p.N; c0 += 4 * T * NV * S) {
            const int64_t at = c0 + (VEC ? 4 * t : t);
            float4 s[NV], r[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                r[i] = p.R ? load4<VEC, T>(p.R + m * p.ldr, at + 4 * T * i, real) : s[i];
            }
            for (int j = 0; j < p.k; j += 2) {  // two choices' rows at a time, added in order
                float4 v[2][NV];
                int64_t row[2];
                float w[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    row[q] = j + q < p.k ? slots.slot(m, j + q) : -1;
                    w[q] = slots.of(m, j + q < p.k ? j + q : j);
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        v[q][i] = load4<VEC, T>(p.A + row[q] * p.lda, at + 4 * T * i, row[q] >= 0 ? p.N : 0);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (row[q] < 0) continue;
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        s[i] = make_float4(fmaf(w[q], v[q][i].x, s[i].x), fmaf(w[q], v[q][i].y, s[i].y),
                                           fmaf(w[q], v[q][i].z, s[i].z), fmaf(w[q], v[q][i].w, s[i].w));
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
                store4<VEC, T>(p.C + m * p.ldc, at + 4 * T * i, real,
                               p.R ? make_float4(s[i].x + r[i].x, s[i].y + r[i].y, s[i].z + r[i].z, s[i].w + r[i].w) : s[i]);
        }
    }
}

// f(T, NV, S) for the sizes.  Few tokens have a block each, whose warps share the
// columns: dispatch, combine, backward of 64 tokens of 4096, k = 8, 19, 22.5 and 29.6
// us with a warp a token, 4.2, 4.7 and 6.1 with a block; 596 of 3104, k = 7, 15.6, 18.2,
// 39.3 and 9.1, 8.1, 20.0; 1000 of 4096, k = 2, 7.6, 10.0, 12.7 and 7.5, 7.5, 11.0, but 1000
// of 256, k = 2, 2.6, 2.3, 3.2 and 3.4, 3.4, 4.6, and 2400 of 2048 8.1, 7.2, 11.5 and
// 8.0, 9.5, 16.7.
template <class F> void for_width(int64_t M, int64_t N, int sm_count, F f) {
    using std::integral_constant;
#define EMU_WIDTH(T, NV, S) f(integral_constant<int, T>{}, integral_constant<int, NV>{}, integral_constant<int, S>{})
    if (N <= 16) EMU_WIDTH(4, 1, 1);
    else if (N <= 32) EMU_WIDTH(8, 1, 1);
    else if (N <= 64) EMU_WIDTH(16, 1, 1);
    else if (N <= 128) EMU_WIDTH(32, 1, 1);
    else if (M <= (N <= 1024 ? 4 : 8) * (int64_t)sm_count) {
        if (N <= 1024) EMU_WIDTH(32, 1, 8);
        else if (N <= 2048) EMU_WIDTH(32, 2, 8);
        else EMU_WIDTH(32, 4, 8);
    }
    else if (N <= 256) EMU_WIDTH(32, 2, 1);
    else EMU_WIDTH(32, 4, 1);
#undef EMU_WIDTH
}

// Blocks per SM: what is resident, in turns of equal length; three for a dispatch
// whose rows are one load, whose writes more of them slow down.  M = 552960, k = 2,
// N = 256, at the copy rate for the bytes of each pass: dispatch 95% (all
// resident: 87%), combine with a residual 96%, backward 96%, dispatch's gradient
// 95%; M = 138241, N = 1024: 88, 91, 101 and 92%; M = 65537, N = 1001 (rows off
// the 16-byte boundaries), k = 4: 81, 85, 96 and 84%; M = 552960, N = 64, k = 8:
// 79, 68, 90 and 67%.
enum Kind { DISPATCH, COMBINE, COMBINE_BWD };

emu_status_t launch(Kind kind, const Exchange& p, emu_stream_t stream) {
    DeviceCtx dev;
    const emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = (p.N & 3) == 0 && vec4_ok(p.A, p.lda) && vec4_ok(p.R, p.R ? p.ldr : 0) && vec4_ok(p.C, p.C ? p.ldc : 0);
    cudaGetLastError();
    for_width(p.M, p.N, dev.sm_count, [&](auto T, auto NV, auto S) {
        constexpr int t = decltype(T)::value, nv = decltype(NV)::value, s_ = decltype(S)::value, tokens = kThreads / t / s_;
        const int64_t groups = (p.M + tokens - 1) / tokens;
        auto run = [&](auto kernel, int per_sm) {
            const int64_t most = (int64_t)dev.sm_count * per_sm, turns = (groups + most - 1) / most;
            kernel<<<(unsigned)((groups + turns - 1) / turns), kThreads, 0, s>>>(p);
        };
        auto go = [&](auto VEC) {
            constexpr bool v = decltype(VEC)::value;
            constexpr auto dispatch = dispatch_kernel<t, nv, s_, v, false>, back = dispatch_kernel<t, nv, s_, v, true>;
            constexpr auto combine = combine_kernel<t, nv, s_, v>;
            static const int resident[3] = {resident_blocks(dispatch, kThreads), resident_blocks(combine, kThreads),
                                            resident_blocks(back, kThreads)};
            if (kind == DISPATCH) run(dispatch, p.N <= 512 && resident[DISPATCH] > 3 ? 3 : resident[DISPATCH]);
            else if (kind == COMBINE) run(combine, resident[COMBINE]);
            else run(back, resident[COMBINE_BWD]);
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
