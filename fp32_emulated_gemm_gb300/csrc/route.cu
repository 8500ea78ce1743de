// route.cu -- the router of a layer of experts: each token's k largest logits,
// their softmax weights and its gradient, and the choices sorted by expert.
//
// Token m with logits l[m, 0..E): its choices are the k largest, the lowest index
// first among equals; a logit of -inf is a closed expert and never chosen, so a
// row may have fewer (expert -1, weight 0, no slot).  Weights are
//   w_j = exp(l_j - l_max) / sum,  the sum over the chosen logits or all of them;
//   dl_e = sum over j with expert e of w_j dw_j - p_e sum_j w_j dw_j,
// p the same softmax (over the chosen: 0 for the others).
//
// Sorted: the choices m k + j in their order, by expert (a stable counting sort):
// offsets[e] is expert e's first row, slots[m, j] choice j's row, sources[row]
// the choice m k + j it came from.  Choices that go nowhere have slot -1, the
// rows behind the last expert's source -1.  Two launches: the choices with a
// histogram for each block of tokens; then every block adds up the histograms
// (of the blocks before it and of all), and places its own choices, ranked among
// their warp's by matching lanes.  Sums of integers alone: no order to depend on.
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace emu {
namespace {

constexpr int kMaxExperts = 1024, kMaxChoices = 32;
constexpr int kThreads = 512, kWarps = kThreads / 32;

struct Route {
    int64_t M;
    int E, k;
    const float* logits;
    int64_t ldl;
    int over_all;
    int32_t* experts;        // M k (sort alone: read)
    float* weights;          // M k
    int32_t *slots, *sources, *offsets;
    int32_t* hist;           // blocks x E
    int64_t rows_per;        // tokens of a block
};

// Logits as integers in their order; NaN above all (it shows in the weight), +0
// and -0 alike.  0 is below every logit: a lane's values that have been taken.
constexpr uint32_t kClosed = 0x007FFFFFu;  // -inf
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key);
}

// The choices and weights of the block's tokens, T lanes a token, which hold V
// logits each (e = lane + T i).  T >= k: lane j keeps choice j.
template <int T, int V> __device__ __forceinline__ void choose(const Route& p, int64_t r0, int64_t r1, int32_t* hist) {
    const int t = threadIdx.x % T;
    for (int64_t base = r0; base < r1; base += kThreads / T) {
        const int64_t m = base + threadIdx.x / T;
        const bool real = m < r1;
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = t + T * i;
            key[i] = real && e < p.E ? order_key(__ldg(p.logits + m * p.ldl + e)) : 0u;
        }
        float top = 0.f, total = 0.f, mine = 0.f;
        int expert = -1;
        for (int j = 0; j < p.k; ++j) {
            uint32_t best = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i] > best) { best = key[i]; at = t + T * i; }
#pragma unroll
            for (int o = T / 2; o > 0; o >>= 1) {
                const uint32_t b = __shfl_xor_sync(0xFFFFFFFFu, best, o);
                const int a = __shfl_xor_sync(0xFFFFFFFFu, at, o);
                if (b > best || (b == best && a < at)) { best = b; at = a; }
            }
            const bool open = best > kClosed;
            const float v = key_value(best);
            if (j == 0) {
                top = open ? v : 0.f;
                if (p.over_all) {
                    // (all of them, while none is taken)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (key[i] > kClosed) total += expf(key_value(key[i]) - top);
#pragma unroll
                    for (int o = T / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
                }
            }
            const float w = open ? expf(v - top) : 0.f;
            if (!p.over_all) total += w;
            if (t == j) { expert = open ? at : -1; mine = w; }
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (t + T * i == at && open) key[i] = 0u;
        }
        if (real && t < p.k) {
            p.experts[m * p.k + t] = expert;
            p.weights[m * p.k + t] = expert >= 0 ? mine / total : 0.f;
            if (expert >= 0) atomicAdd(&hist[expert], 1);
        }
    }
}

// T and V for E experts: few lanes, so that a warp has many tokens and little to
// exchange, but at least a lane for each choice.
#define EMU_LANES(T, V) choose<T, V>(p, r0, r1, hist)
__device__ __forceinline__ void choose_any(const Route& p, int64_t r0, int64_t r1, int32_t* hist) {
    const int lanes = p.k > (p.E + 3) / 4 ? p.k : (p.E + 3) / 4;
    if (lanes <= 4) EMU_LANES(4, 4);
    else if (lanes <= 8) EMU_LANES(8, 4);
    else if (lanes <= 16) EMU_LANES(16, 4);
    else if (p.E <= 128) EMU_LANES(32, 4);
    else if (p.E <= 256) EMU_LANES(32, 8);
    else if (p.E <= 512) EMU_LANES(32, 16);
    else EMU_LANES(32, 32);
}
#undef EMU_LANES

// Where the block's choices [c0, c1) go.  `count[w][e]` becomes the next row of
// expert e for warp w; `first[e]` comes with the row of the block's first choice
// of expert e.
__device__ __forceinline__ void place(const Route& p, int64_t c0, int64_t c1, const int32_t* first, int32_t* count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t per = ((c1 - c0 + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int64_t w0 = c0 + warp * per, w1 = w0 + per < c1 ? w0 + per : c1;
    int32_t* mine = count + warp * p.E;
    for (int i = threadIdx.x; i < kWarps * p.E; i += kThreads) count[i] = 0;
    __syncthreads();
    for (int64_t c = w0 + lane; c < w1; c += 32) {
        const int e = p.experts[c];
        if ((unsigned)e < (unsigned)p.E) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        int32_t at = first[e];
        for (int w = 0; w < kWarps; ++w) {
            const int32_t n = count[w * p.E + e];
            count[w * p.E + e] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int64_t c = w0; c < w1; c += 32) {
        const int64_t i = c + lane;
        int e = i < w1 ? p.experts[i] : -1;
        if ((unsigned)e >= (unsigned)p.E) e = -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int32_t row = -1;
        if (e >= 0) row = mine[e] + rank;
        __syncwarp();
        if (e >= 0 && rank == 0) mine[e] += __popc(same);
        __syncwarp();
        if (i < w1) {
            p.slots[i] = row;
            if (row >= 0) p.sources[row] = (int32_t)i;
        }
    }
}

// Exclusive sums of total[0..E) by the block: start[e], and start[E] the sum.
__device__ __forceinline__ void exclusive_sums(const int32_t* total, int32_t* start, int E) {
    // a warp does it: E / 32 steps
    if (threadIdx.x < 32) {
        int32_t carry = 0;
        for (int base = 0; base < E; base += 32) {
            const int e = base + threadIdx.x;
            const int32_t n = e < E ? total[e] : 0;
            int32_t s = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t up = __shfl_up_sync(0xFFFFFFFFu, s, o);
                if (threadIdx.x >= o) s += up;
            }
            if (e < E) start[e] = carry + s - n;
            carry += __shfl_sync(0xFFFFFFFFu, s, 31);
        }
        if (threadIdx.x == 0) start[E] = carry;
    }
    __syncthreads();
}

// Shared memory of a block: histogram, starts and the warps' counts.
size_t smem_of(int E) { return (size_t)((kWarps + 2) * E + 1) * sizeof(int32_t); }

// Choices (or, SORT, their histogram alone) of the block's tokens.
template <bool SORT> __global__ void __launch_bounds__(kThreads) choose_kernel(const __grid_constant__ Route p) {
    extern __shared__ int32_t sh[];
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int64_t r0 = blockIdx.x * p.rows_per, r1 = r0 + p.rows_per < p.M ? r0 + p.rows_per : p.M;
    for (int e = threadIdx.x; e < p.E; e += kThreads) sh[e] = 0;
    __syncthreads();
    if constexpr (SORT) {
        for (int64_t c = r0 * p.k + threadIdx.x; c < r1 * p.k; c += kThreads) {
            const int e = p.experts[c];
            if ((unsigned)e < (unsigned)p.E) atomicAdd(&sh[e], 1);
        }
    } else {
        choose_any(p, r0, r1, sh);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kThreads) p.hist[(int64_t)blockIdx.x * p.E + e] = sh[e];
}

__global__ void __launch_bounds__(kThreads) place_kernel(const __grid_constant__ Route p) {
    extern __shared__ int32_t sh[];
    int32_t *total = sh, *start = sh + p.E, *count = start + p.E + 1, *before = count;  // (before's place is count's)
    for (int e = threadIdx.x; e < p.E; e += kThreads) { total[e] = 0; before[e] = 0; }
    __syncthreads();
    griddep_wait();
    // the threads share the histograms: expert by expert within a row of them
    const int64_t n = (int64_t)gridDim.x * p.E, mine = (int64_t)blockIdx.x * p.E;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const int32_t h = p.hist[i];
        if (h == 0) continue;
        const int e = (int)(i % p.E);
        atomicAdd(&total[e], h);
        if (i < mine) atomicAdd(&before[e], h);
    }
    __syncthreads();
    exclusive_sums(total, start, p.E);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = start[e];
    const int64_t C = p.M * p.k, last = start[p.E];
    for (int64_t i = last + blockIdx.x * (int64_t)kThreads + threadIdx.x; i < C; i += (int64_t)gridDim.x * kThreads)
        p.sources[i] = -1;
    for (int e = threadIdx.x; e < p.E; e += kThreads) total[e] = start[e] + before[e];
    __syncthreads();
    const int64_t r0 = blockIdx.x * p.rows_per, r1 = r0 + p.rows_per < p.M ? r0 + p.rows_per : p.M;
    place(p, r0 * p.k, r1 * p.k, total, count);
}

// A few tokens: one block does both.
template <bool SORT> __global__ void __launch_bounds__(kThreads) route_small_kernel(const __grid_constant__ Route p) {
    extern __shared__ int32_t sh[];
    int32_t *total = sh, *start = sh + p.E, *count = start + p.E + 1;
    for (int e = threadIdx.x; e < p.E; e += kThreads) total[e] = 0;
    __syncthreads();
    const int64_t C = p.M * p.k;
    if constexpr (SORT) {
        for (int64_t c = threadIdx.x; c < C; c += kThreads) {
            const int e = p.experts[c];
            if ((unsigned)e < (unsigned)p.E) atomicAdd(&total[e], 1);
        }
    } else {
        choose_any(p, 0, p.M, total);
    }
    __syncthreads();
    exclusive_sums(total, start, p.E);
    for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = start[e];
    for (int64_t i = start[p.E] + threadIdx.x; i < C; i += kThreads) p.sources[i] = -1;
    place(p, 0, C, start, count);
}

// dlogits, T lanes a token (T >= k: lane j holds choice j).
struct RouteBwd {
    int64_t M;
    int E, k;
    const float *dweights, *logits;
    int64_t ldl;
    const int32_t* experts;
    const float* weights;
    int over_all;
    float* dlogits;
    int64_t lddl;
};
template <int T> __global__ void __launch_bounds__(256) route_bwd_kernel(const __grid_constant__ RouteBwd p) {
    const int t = threadIdx.x % T;
    const int64_t step = (int64_t)gridDim.x * (256 / T);
    for (int64_t base = blockIdx.x * (int64_t)(256 / T); base < p.M; base += step) {
        const int64_t m = base + threadIdx.x / T;
        const bool real = m < p.M;
        int e = -1;
        float g = 0.f, w = 0.f;
        if (real && t < p.k) {
            e = p.experts[m * p.k + t];
            w = p.weights[m * p.k + t];
            if (e >= 0) g = w * p.dweights[m * p.k + t];
        }
        float inner = g;
#pragma unroll
        for (int o = T / 2; o > 0; o >>= 1) inner += __shfl_xor_sync(0xFFFFFFFFu, inner, o);
        // over the chosen: w_j (dw_j - inner) for them, 0 elsewhere
        if (!p.over_all) g = fmaf(-w, inner, g);
        // over all: p_e = exp(l_e - l_first) w_first, and w_first is the largest
        const int e0 = __shfl_sync(0xFFFFFFFFu, e, 0, T);
        const float w0 = __shfl_sync(0xFFFFFFFFu, w, 0, T);
        const bool all = p.over_all && real && e0 >= 0 && e0 < p.E;
        const float l0 = all ? __ldg(p.logits + m * p.ldl + e0) : 0.f;
        for (int first = 0; first < p.E; first += T) {
            const int c = first + t;
            float d = 0.f;
            if (all && c < p.E) {
                const float l = __ldg(p.logits + m * p.ldl + c);
                d = l == -INFINITY ? 0.f : -expf(l - l0) * w0 * inner;
            }
            for (int j = 0; j < p.k; ++j) {
                const int ej = __shfl_sync(0xFFFFFFFFu, e, j, T);
                const float gj = __shfl_sync(0xFFFFFFFFu, g, j, T);
                if (ej == c) d += gj;
            }
            if (real && c < p.E) p.dlogits[m * p.lddl + c] = d;
        }
    }
}

// One block for as much as it does in the time that a second launch takes.
constexpr int64_t kSmallLogits = 8192;

bool sizes_ok(int64_t M, int E, int k) {
    return E <= kMaxExperts && k <= kMaxChoices && M <= (INT32_MAX - 256) / (k > 0 ? k : 1);
}

template <bool SORT> emu_status_t route(Route p, emu_stream_t stream) {
    DeviceCtx dev;
    emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = smem_of(p.E);
    const StreamLock lock(s);
    cudaGetLastError();
    if (p.M * (SORT ? p.k : p.E) <= kSmallLogits) {
        static const cudaError_t attr =
            cudaFuncSetAttribute(route_small_kernel<SORT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(kMaxExperts));
        if (attr != cudaSuccess) return EMU_STATUS_LAUNCH_FAILED;
        route_small_kernel<SORT><<<1, kThreads, smem, s>>>(p);
        return cudaGetLastError() == cudaSuccess ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED;
    }
    static const cudaError_t attr =
        cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(kMaxExperts));
    if (attr != cudaSuccess) return EMU_STATUS_LAUNCH_FAILED;
    int64_t blocks = (p.M + 63) / 64;
    if (blocks > dev.sm_count) blocks = dev.sm_count;
    p.rows_per = (p.M + blocks - 1) / blocks;
    blocks = (p.M + p.rows_per - 1) / p.rows_per;
    float* scratch = nullptr;
    st = reduce_scratch(dev.id, s, (size_t)blocks * p.E, &scratch);
    if (st != EMU_STATUS_SUCCESS) return st;
    p.hist = reinterpret_cast<int32_t*>(scratch);
    choose_kernel<SORT><<<(unsigned)blocks, kThreads, p.E * sizeof(int32_t), s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return EMU_STATUS_LAUNCH_FAILED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = la;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, place_kernel, p) != cudaSuccess) {
        cudaGetLastError();
        return EMU_STATUS_LAUNCH_FAILED;
    }
    return EMU_STATUS_SUCCESS;
}

emu_status_t no_tokens(int E, int32_t* offsets, emu_stream_t stream) {
    if (!offsets) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev;
    const emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    if (cudaMemsetAsync(offsets, 0, (size_t)(E + 1) * sizeof(int32_t), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess)
        return EMU_STATUS_SUCCESS;
    cudaGetLastError();
    return EMU_STATUS_LAUNCH_FAILED;
}

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" {

emu_status_t emu_expert_route(emu_over_t over, int64_t M, int E, int k, const float* logits, int64_t ldl, int32_t* experts,
                              float* weights, int32_t* slots, int32_t* sources, int32_t* offsets, emu_stream_t stream) {
    if ((over != EMU_OVER_CHOSEN && over != EMU_OVER_ALL) || M < 0 || E < 1 || k < 1 || k > E) return EMU_STATUS_INVALID_VALUE;
    if (!sizes_ok(M, E, k)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0) return no_tokens(E, offsets, stream);
    if (!logits || ldl < E || !experts || !weights || !slots || !sources || !offsets) return EMU_STATUS_INVALID_VALUE;
    return route<false>({M, E, k, logits, ldl, over == EMU_OVER_ALL, experts, weights, slots, sources, offsets, nullptr, 0},
                        stream);
}

emu_status_t emu_expert_sort(int64_t M, int E, int k, const int32_t* experts, int32_t* slots, int32_t* sources,
                             int32_t* offsets, emu_stream_t stream) {
    if (M < 0 || E < 1 || k < 1) return EMU_STATUS_INVALID_VALUE;
    if (!sizes_ok(M, E, k)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0) return no_tokens(E, offsets, stream);
    if (!experts || !slots || !sources || !offsets) return EMU_STATUS_INVALID_VALUE;
    return route<true>({M, E, k, nullptr, 0, 0, const_cast<int32_t*>(experts), nullptr, slots, sources, offsets, nullptr, 0},
                       stream);
}

emu_status_t emu_expert_route_bwd(emu_over_t over, int64_t M, int E, int k, const float* dweights, const float* logits,
                                  int64_t ldl, const int32_t* experts, const float* weights, float* dlogits, int64_t lddl,
                                  emu_stream_t stream) {
    if ((over != EMU_OVER_CHOSEN && over != EMU_OVER_ALL) || M < 0 || E < 1 || k < 1 || k > E) return EMU_STATUS_INVALID_VALUE;
    if (!sizes_ok(M, E, k)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0) return EMU_STATUS_SUCCESS;
    if (!dweights || !experts || !weights || !dlogits || lddl < E) return EMU_STATUS_INVALID_VALUE;
    if (over == EMU_OVER_ALL && (!logits || ldl < E)) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev;
    const emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const RouteBwd p{M, E, k, dweights, logits, ldl, experts, weights, over == EMU_OVER_ALL, dlogits, lddl};
    const int lanes = k > E ? k : (E < 32 ? E : 32);
    cudaGetLastError();
    auto launch = [&](auto kernel, int T) {
        const int64_t groups = (M + 256 / T - 1) / (256 / T), most = (int64_t)dev.sm_count * 8;
        kernel<<<(unsigned)(groups < most ? groups : most), 256, 0, s>>>(p);
    };
    if (lanes <= 4) launch(route_bwd_kernel<4>, 4);
    else if (lanes <= 8) launch(route_bwd_kernel<8>, 8);
    else if (lanes <= 16) launch(route_bwd_kernel<16>, 16);
    else launch(route_bwd_kernel<32>, 32);
    return cudaGetLastError() == cudaSuccess ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED;
}

}  // extern "C"
