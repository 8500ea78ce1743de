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
// M = 552960, E = 16, k = 2 (forward 53 MB, backward 49): 25.8 and 10.5 us, 7.8 and
// 7.2 at the copy rate; the choice is bound by its instructions, the sort by its
// two passes over the choices and the scattered words of `sources`.
#include <cuda_runtime.h>

#include "internal.h"
#include "norm_rows.cuh"

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
    int32_t* hist;           // choosing blocks x E
    int hists;
    int64_t rows_per;        // tokens of a choosing block
    int per_place;           // choosing blocks whose choices a placing block has
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

// The choices and weights of the block's tokens [r0, r1), T lanes a token (1 or 8):
// each goes through its share of the logits with the K (>= k) largest so far in
// order; the lanes' lists are then merged choice by choice.
template <int K, int T> __device__ __forceinline__ void choose_lists(const Route& p, int64_t r0, int64_t r1, int32_t* hist) {
    const bool vec = (p.E & 3) == 0 && (p.ldl & 3) == 0 && (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0;
    const int t = threadIdx.x % T;
    for (int64_t base = r0; base < r1; base += kThreads / T) {
        const int64_t m = base + threadIdx.x / T;
        const bool real = m < r1;
        const float* row = p.logits + (real ? m : r0) * p.ldl;
        uint32_t key[K];
        int at[K];
#pragma unroll
        for (int j = 0; j < K; ++j) { key[j] = kClosed; at[j] = -1; }  // (a closed logit is not above it)
        auto insert = [&](float v, int e) {
            const uint32_t x = order_key(v);
            if (x <= key[K - 1]) return;
#pragma unroll
            for (int j = K - 1; j > 0; --j) {
                if (x > key[j - 1]) { key[j] = key[j - 1]; at[j] = at[j - 1]; }
                else if (x > key[j]) { key[j] = x; at[j] = e; }
            }
            if (x > key[0]) { key[0] = x; at[0] = e; }
        };
        if (vec) {
#pragma unroll 4
            for (int e = 4 * t; e < p.E; e += 4 * T) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(row + e));
                insert(v.x, e);
                insert(v.y, e + 1);
                insert(v.z, e + 2);
                insert(v.w, e + 3);
            }
        } else {
#pragma unroll 8
            for (int e = t; e < p.E; e += T) insert(__ldg(row + e), e);
        }
        if constexpr (T > 1) {
            // the lists' first elements: the largest, then the lowest index; its lane
            // moves on
            uint32_t out_key[K];
            int out_at[K];
#pragma unroll
            for (int j = 0; j < K; ++j) {
                uint32_t best = key[0];
                int e = at[0];
#pragma unroll
                for (int o = T / 2; o > 0; o >>= 1) {
                    const uint32_t b = __shfl_xor_sync(0xFFFFFFFFu, best, o);
                    const int f = __shfl_xor_sync(0xFFFFFFFFu, e, o);
                    if (b > best || (b == best && f < e)) { best = b; e = f; }
                }
                out_key[j] = best;
                out_at[j] = e;
                if (at[0] == e) {
#pragma unroll
                    for (int i = 0; i + 1 < K; ++i) { key[i] = key[i + 1]; at[i] = at[i + 1]; }
                    key[K - 1] = kClosed;
                    at[K - 1] = -1;
                }
            }
#pragma unroll
            for (int j = 0; j < K; ++j) { key[j] = out_key[j]; at[j] = out_at[j]; }
        }
        const float top = at[0] >= 0 ? key_value(key[0]) : 0.f;
        float w[K], total = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            w[j] = at[j] >= 0 ? expf(key_value(key[j]) - top) : 0.f;
            if (j < p.k) total += w[j];
        }
        if (p.over_all) {
            total = 0.f;
#pragma unroll 4
            for (int e = t; e < p.E; e += T) total += expf(__ldg(row + e) - top);  // (exp(-inf) = 0)
#pragma unroll
            for (int o = T / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        }
        if (!real) continue;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (j < p.k && j % T == t) {
                p.experts[m * p.k + j] = at[j];
                p.weights[m * p.k + j] = at[j] >= 0 ? w[j] / total : 0.f;
                if (at[j] >= 0) atomicAdd(&hist[at[j]], 1);
            }
    }
}

// Likewise with T lanes a token, which hold V logits each (e = lane + T i) and find
// the choices one by one.  T >= k: lane j keeps choice j.
template <int T, int V> __device__ __forceinline__ void choose_lanes(const Route& p, int64_t r0, int64_t r1, int32_t* hist) {
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

// Which of the two, and its sizes (a kernel each: what holds 32 logits a thread
// would cost the others their occupancy).
enum Way { SORT, LIST_1, LIST_2, LIST_4, LIST_8, SHARED_1, SHARED_2, SHARED_4, SHARED_8, LANES_4, LANES_8, LANES_16, LANES_32 };
template <int WAY> __device__ __forceinline__ void choose(const Route& p, int64_t r0, int64_t r1, int32_t* hist) {
    if constexpr (WAY == SORT) {
        for (int64_t c = r0 * p.k + threadIdx.x; c < r1 * p.k; c += kThreads) {
            const int e = p.experts[c];
            if ((unsigned)e < (unsigned)p.E) atomicAdd(&hist[e], 1);
        }
    } else if constexpr (WAY < SHARED_1) {
        choose_lists<1 << (WAY - LIST_1), 1>(p, r0, r1, hist);
    } else if constexpr (WAY < LANES_4) {
        choose_lists<1 << (WAY - SHARED_1), 8>(p, r0, r1, hist);
    } else {
        choose_lanes<32, 4 << (WAY - LANES_4)>(p, r0, r1, hist);
    }
}
constexpr int tokens_of(int way) { return way < SHARED_1 ? kThreads : way < LANES_4 ? kThreads / 8 : kThreads / 32; }
// A lane a token needs the fewest instructions, which bound it, and many tokens;
// with few, eight lanes share the wait for one.  Route and sort, a lane / eight:
// M = 552960, E = 16, k = 2 25.8 / 57 us (one lane for all four of 16 logits and a
// search of them for each choice: 49 us); 138240, 64, 8 56 / 80; 34560, 256, 8 55 /
// 66; 6144, 64, 8 25 / 12; 8000, 1024, 4 91 / 43; 1000, 128, 8 35 / 12.8.  Lists of
// more than eight would not fit a lane's registers; there a search for each choice
// takes a warp a token.
constexpr int64_t kSharedTokens = 20000;
Way way_of(int64_t M, int E, int k) {
    if (k <= 8) return Way((M < kSharedTokens ? SHARED_1 : LIST_1) + (k == 1 ? 0 : k == 2 ? 1 : k <= 4 ? 2 : 3));
    return E <= 128 ? LANES_4 : E <= 256 ? LANES_8 : E <= 512 ? LANES_16 : LANES_32;
}

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
#pragma unroll 4
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
    int next = w0 + lane < w1 ? p.experts[w0 + lane] : -1;
    for (int64_t c = w0; c < w1; c += 32) {
        const int64_t i = c + lane;
        int e = next;
        next = i + 32 < w1 ? p.experts[i + 32] : -1;
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

template <int WAY> __global__ void __launch_bounds__(kThreads) choose_kernel(const __grid_constant__ Route p) {
    extern __shared__ int32_t sh[];
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int64_t r0 = blockIdx.x * p.rows_per, r1 = r0 + p.rows_per < p.M ? r0 + p.rows_per : p.M;
    for (int e = threadIdx.x; e < p.E; e += kThreads) sh[e] = 0;
    __syncthreads();
    choose<WAY>(p, r0, r1, sh);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kThreads) p.hist[(int64_t)blockIdx.x * p.E + e] = sh[e];
}

__global__ void __launch_bounds__(kThreads) place_kernel(const __grid_constant__ Route p) {
    extern __shared__ int32_t sh[];
    int32_t *total = sh, *start = sh + p.E, *count = start + p.E + 1, *before = count;  // (before's place is count's)
    for (int e = threadIdx.x; e < p.E; e += kThreads) { total[e] = 0; before[e] = 0; }
    __syncthreads();
    griddep_wait();
    // the threads share the histograms: some threads an expert, a sum each
    const int parts = p.E < kThreads ? kThreads / p.E : 1, wide = kThreads / parts;
    const int mine = blockIdx.x * p.per_place;
    for (int e = threadIdx.x % wide, part = threadIdx.x / wide; e < p.E && part < parts; e += wide) {
        int32_t all = 0, ahead = 0;
        for (int b = part; b < p.hists; b += 16 * parts) {  // sixteen loads at a time
            int32_t h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) h[i] = b + i * parts < p.hists ? __ldcg(p.hist + (int64_t)(b + i * parts) * p.E + e) : 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                all += h[i];
                if (b + i * parts < mine) ahead += h[i];
            }
        }
        atomicAdd(&total[e], all);
        atomicAdd(&before[e], ahead);
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
    const int64_t per = p.per_place * p.rows_per, r0 = blockIdx.x * per, r1 = r0 + per < p.M ? r0 + per : p.M;
    place(p, r0 * p.k, r1 * p.k, total, count);
}

// A few tokens: one block does both.
template <int WAY> __global__ void __launch_bounds__(kThreads) route_small_kernel(const __grid_constant__ Route p) {
    extern __shared__ int32_t sh[];
    int32_t *total = sh, *start = sh + p.E, *count = start + p.E + 1;
    for (int e = threadIdx.x; e < p.E; e += kThreads) total[e] = 0;
    __syncthreads();
    const int64_t C = p.M * p.k;
    choose<WAY>(p, 0, p.M, total);
    __syncthreads();
    exclusive_sums(total, start, p.E);
    for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = start[e];
    for (int64_t i = start[p.E] + threadIdx.x; i < C; i += kThreads) p.sources[i] = -1;
    place(p, 0, C, start, count);
}

// dlogits: a thread has eight columns of a token and works out the token's sum for
// itself (the choices' words are few, and in L1 for all but the first of them).
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
template <bool VEC, int K> __global__ void __launch_bounds__(256) route_bwd_kernel(const __grid_constant__ RouteBwd p) {
    constexpr int C = 8;
    const uint32_t quads = (p.E + C - 1) / C;
    const int64_t n = p.M * quads, step = (int64_t)gridDim.x * 256;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += step) {
        const int64_t m = n <= UINT32_MAX ? (uint32_t)i / quads : i / quads;
        const int c = C * (int)(i - m * quads);
        const int32_t* experts = p.experts + m * p.k;
        const float *weights = p.weights + m * p.k, *dweights = p.dweights + m * p.k;
        float d[C] = {}, inner = 0.f;
        int at[K], e0 = -1;
        float w[K], g[K], w0 = 0.f;
        // (K choices at a time, whose loads go out together)
        auto load = [&](int j0) {
#pragma unroll
            for (int j = 0; j < K; ++j) {
                const bool there = j0 + j < p.k;
                at[j] = there ? __ldg(experts + j0 + j) : -1;
                w[j] = there ? __ldg(weights + j0 + j) : 0.f;
                g[j] = there ? __ldg(dweights + j0 + j) : 0.f;
            }
        };
        for (int j0 = 0; j0 < p.k; j0 += K) {
            load(j0);
            if (j0 == 0) { e0 = at[0]; w0 = w[0]; }
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (at[j] >= 0) inner = fmaf(w[j], g[j], inner);
        }
        if (p.over_all && e0 >= 0 && e0 < p.E) {
            // p_e = exp(l_e - l_first) w_first, and w_first is the largest
            const float l0 = __ldg(p.logits + m * p.ldl + e0);
            const float4 l = load4<VEC, 1>(p.logits + m * p.ldl, c, p.E), h = load4<VEC, 1>(p.logits + m * p.ldl, c + 4, p.E);
            const float v[C] = {l.x, l.y, l.z, l.w, h.x, h.y, h.z, h.w};
#pragma unroll
            for (int q = 0; q < C; ++q) d[q] = v[q] == -INFINITY ? 0.f : -expf(v[q] - l0) * w0 * inner;
        }
        for (int j0 = 0; j0 < p.k; j0 += K) {
            if (p.k > K) load(j0);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                // over the chosen: w_j (dw_j - inner) for them, 0 elsewhere
                const float s = w[j] * (p.over_all ? g[j] : g[j] - inner);
#pragma unroll
                for (int q = 0; q < C; ++q)
                    if (at[j] == c + q) d[q] += s;
            }
        }
        store4<VEC, 1>(p.dlogits + m * p.lddl, c, p.E, make_float4(d[0], d[1], d[2], d[3]));
        store4<VEC, 1>(p.dlogits + m * p.lddl, c + 4, p.E, make_float4(d[4], d[5], d[6], d[7]));
    }
}

// One block for as much as it does in the time that a second launch takes (1000
// tokens of 8 choices: sorted by one block 13.8 us).
constexpr int64_t kSmallLogits = 8192, kSmallChoices = 2048;

bool sizes_ok(int64_t M, int E, int k) {
    return E <= kMaxExperts && k <= kMaxChoices && M <= (INT32_MAX - 256) / (k > 0 ? k : 1);
}

// What a launch may have without being asked for is 48 KB (682 experts); beyond it
// the current device is asked, call by call, for the most that any call needs: the
// limit is the kernel's, and another thread's call with fewer experts must not lower
// it between this one's request and its launch.
template <class K> emu_status_t allow_smem(K kernel, size_t bytes) {
    if (bytes <= 48 * 1024) return EMU_STATUS_SUCCESS;
    return launched(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(kMaxExperts)));
}

template <int WAY> emu_status_t route(Route p, emu_stream_t stream) {
    DeviceCtx dev;
    emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = smem_of(p.E);
    const StreamLock lock(s);
    if (p.M * p.k <= kSmallChoices && (WAY == SORT || p.M * p.E <= kSmallLogits)) {
        EMU_TRY(allow_smem(route_small_kernel<WAY>, smem));
        cudaGetLastError();
        route_small_kernel<WAY><<<1, kThreads, smem, s>>>(p);
        return launched(cudaGetLastError());
    }
    static const int resident = resident_blocks(choose_kernel<WAY>, kThreads);
    EMU_TRY(allow_smem(place_kernel, smem));
    // choosing: a pass over the tokens that are resident at once, or several of equal
    // length; placing: no more blocks than keep the histograms, which each of them
    // reads, fewer than the choices
    const int64_t choosers = even_grid(p.M, tokens_of(WAY), (int64_t)dev.sm_count * resident);
    p.rows_per = (p.M + choosers - 1) / choosers;
    p.hists = (int)((p.M + p.rows_per - 1) / p.rows_per);
    int64_t placers = p.M * p.k / (4 * (int64_t)p.E);
    placers = placers < 1 ? 1 : placers > p.hists ? p.hists : placers;
    p.per_place = (int)((p.hists + placers - 1) / placers);
    placers = (p.hists + p.per_place - 1) / p.per_place;
    float* scratch = nullptr;
    EMU_TRY(reduce_scratch(dev.id, s, (size_t)p.hists * p.E, &scratch));
    p.hist = reinterpret_cast<int32_t*>(scratch);
    cudaGetLastError();
    choose_kernel<WAY><<<(unsigned)p.hists, kThreads, p.E * sizeof(int32_t), s>>>(p);
    EMU_TRY(launched(cudaGetLastError()));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)placers, 1, 1);
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
    const Route p{M, E, k, logits, ldl, over == EMU_OVER_ALL, experts, weights, slots, sources, offsets, nullptr, 0, 0, 0};
    switch (way_of(M, E, k)) {
        case LIST_1: return route<LIST_1>(p, stream);
        case LIST_2: return route<LIST_2>(p, stream);
        case LIST_4: return route<LIST_4>(p, stream);
        case LIST_8: return route<LIST_8>(p, stream);
        case SHARED_1: return route<SHARED_1>(p, stream);
        case SHARED_2: return route<SHARED_2>(p, stream);
        case SHARED_4: return route<SHARED_4>(p, stream);
        case SHARED_8: return route<SHARED_8>(p, stream);
        case LANES_4: return route<LANES_4>(p, stream);
        case LANES_8: return route<LANES_8>(p, stream);
        case LANES_16: return route<LANES_16>(p, stream);
        default: return route<LANES_32>(p, stream);
    }
}

emu_status_t emu_expert_sort(int64_t M, int E, int k, const int32_t* experts, int32_t* slots, int32_t* sources,
                             int32_t* offsets, emu_stream_t stream) {
    if (M < 0 || E < 1 || k < 1) return EMU_STATUS_INVALID_VALUE;
    if (!sizes_ok(M, E, k)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0) return no_tokens(E, offsets, stream);
    if (!experts || !slots || !sources || !offsets) return EMU_STATUS_INVALID_VALUE;
    return route<SORT>({M, E, k, nullptr, 0, 0, const_cast<int32_t*>(experts), nullptr, slots, sources, offsets, nullptr, 0, 0,
                        0}, stream);
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
    const bool vec = (E & 3) == 0 && vec4_ok(dlogits, lddl) && (over != EMU_OVER_ALL || vec4_ok(logits, ldl));
    const int64_t groups = (M * ((E + 7) / 8) + 255) / 256, most = (int64_t)dev.sm_count * 8;
    const unsigned grid = (unsigned)(groups < most ? groups : most);
    cudaGetLastError();
    if (k <= 2) {
        if (vec) route_bwd_kernel<true, 2><<<grid, 256, 0, s>>>(p);
        else route_bwd_kernel<false, 2><<<grid, 256, 0, s>>>(p);
    } else {
        if (vec) route_bwd_kernel<true, 8><<<grid, 256, 0, s>>>(p);
        else route_bwd_kernel<false, 8><<<grid, 256, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED;
}

}  // extern "C"
