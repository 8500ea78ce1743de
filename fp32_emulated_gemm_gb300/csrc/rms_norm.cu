// rms_norm.cu -- root-mean-square norm over the rows of an FP32 matrix after the
// addition of a residual, with an output in FP32 or in 8 bits with scales, and
// its backward pass.
//
// Row s = x + q of width N (q the residual): r = 1 / sqrt(sum s^2 / N + eps),
// h = s r, y = h w.  Backward, with g = dy w:
//   ds = r (g - h mean(g h)) (+ add),  dw = sum over rows of dy h.
// 8 bits: each 128 columns share a scale, the smallest power of two f with
// max |y| <= 448 f (448: the largest e4m3 number), and hold y / f rounded to
// e4m3.  A power of two makes the division exact, so the only rounding beyond
// FP32's is e4m3's own, and costs no precision: e4m3 is a floating format, the
// scale only has to keep it in range.
//
// Bound by memory: the sum needs one pass, the rows stay in registers.  The threads'
// sums of squares are added in two FP32 words, so that a row's mean is off by little
// more than its rounding: what lies next to one of e4m3's borders is rounded by the
// last bit of r.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"
#include "norm_rows.cuh"

namespace emu {
namespace {

constexpr int kGroup = 128;  // columns that share a scale

struct RmsFwd {
    int64_t M, N;
    const float* X;
    int64_t ldx;
    const float* R;  // may be null
    int64_t ldr;
    const float* w;  // may be null
    float eps;
    float* S;        // x + q; null when it is not wanted
    int64_t lds;
    float* rstd;     // may be null
    float* Y;        // FP32 output
    int64_t ldy;
    uint8_t* Q;      // 8-bit output
    int64_t ldq;
    float* scales;
    int64_t ldscales;
};

// A row's columns: thread t of T holds columns c + S j, j = 0..3, of each of its
// NV float4 (VEC: c + j), c = first_col + 4 T i.  Lanes of a warp hold 128
// neighbouring columns at either alignment, so a scale's group is a warp's.
template <int T> constexpr int kStride = T < 32 ? T : 32;
template <int T, bool VEC> __device__ __forceinline__ int64_t first_col(int t, int i) {
    return (VEC ? 4 * t : T <= 32 ? t : kGroup * (t / 32) + t % 32) + (int64_t)4 * T * i;
}

// a + b and what its rounding leaves (Knuth's two-sum).
__device__ __forceinline__ float2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}
// The sum over the T threads of a row of v + low, in two words until the last
// rounding (none of a sum that is infinite or NaN, whose second word is NaN).  `flip`:
// as for row_sum2.
template <int T> __device__ __forceinline__ float row_sum_exact(float v, float low, int& flip) {
    auto add = [&](float hi, float lo) {
        const float2 s = two_sum(v, hi);
        v = s.x;
        low += lo + s.y;
    };
#pragma unroll
    for (int o = T < 32 ? T / 2 : 16; o > 0; o >>= 1) {
        const float hi = __shfl_xor_sync(0xFFFFFFFFu, v, o), lo = __shfl_xor_sync(0xFFFFFFFFu, low, o);
        add(hi, lo);
    }
    if constexpr (T > 32) {
        __shared__ float2 part[2][T / 32];
        float2* p = part[flip];
        flip ^= 1;
        if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = make_float2(v, low);
        __syncthreads();
        v = p[0].x;
        low = p[0].y;
#pragma unroll
        for (int i = 1; i < T / 32; ++i) add(p[i].x, p[i].y);
    }
    return fabsf(v) < INFINITY ? v + low : v;
}
__device__ __forceinline__ float rstd_of(float sum, float inv_n, float eps) {
    return 1.0f / sqrtf(__fadd_rn(__fmul_rn(sum, inv_n), eps));
}

__device__ __forceinline__ float max4(const float4& v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}
// The exponent of the smallest power of two f >= 2^-126 with top <= 448 f
// (448 = 1.75 2^8).
__device__ __forceinline__ int scale_exponent(float top) {
    const uint32_t u = __float_as_uint(top);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < -126 ? -126 : e;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t e4m3x4(const float4& v, float f) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v.x * f, v.y * f), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v.z * f, v.w * f), __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)lo | (uint32_t)hi << 16;
}
template <bool VEC, int S>
__device__ __forceinline__ void store_bytes(uint8_t* row, int64_t c, int64_t n, uint32_t v) {
    if constexpr (VEC) {
        if (c < n) *reinterpret_cast<uint32_t*>(row + c) = v;
    } else {
        if (c < n) row[c] = (uint8_t)v;
        if (c + S < n) row[c + S] = (uint8_t)(v >> 8);
        if (c + 2 * S < n) row[c + 2 * S] = (uint8_t)(v >> 16);
        if (c + 3 * S < n) row[c + 3 * S] = (uint8_t)(v >> 24);
    }
}

template <int T, int NV, bool VEC, bool QUANT>
__global__ void __launch_bounds__(kBlockThreads<T>) rms_fwd_regs_kernel(const __grid_constant__ RmsFwd p) {
    constexpr int G = kBlockRows<T>, S = kStride<T>;
    const int t = threadIdx.x % T, g = threadIdx.x / T;
    const float inv_n = 1.0f / (float)p.N;
    const int64_t step = (int64_t)gridDim.x * G;
    int flip = 0;
    // (the loop is the same for all threads of a block: shuffles and barriers)
    for (int64_t first = blockIdx.x * (int64_t)G; first < p.M; first += step) {
        const int64_t r = first + g;
        const bool real = r < p.M;
        const int64_t n = real ? p.N : 0;
        float4 x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = load4<VEC, S>(p.X + r * p.ldx, first_col<T, VEC>(t, i), n);
        if (p.R) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float4 q = load4<VEC, S>(p.R + r * p.ldr, first_col<T, VEC>(t, i), n);
                x[i] = make_float4(x[i].x + q.x, x[i].y + q.y, x[i].z + q.z, x[i].w + q.w);
            }
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) s += fmaf(x[i].x, x[i].x, x[i].y * x[i].y) + fmaf(x[i].z, x[i].z, x[i].w * x[i].w);
        const float rs = rstd_of(row_sum_exact<T>(s, 0.f, flip), inv_n, p.eps);
        if (p.S) {
#pragma unroll
            for (int i = 0; i < NV; ++i) store4<VEC, S>(p.S + r * p.lds, first_col<T, VEC>(t, i), n, x[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = first_col<T, VEC>(t, i);
            float4 v = make_float4(x[i].x * rs, x[i].y * rs, x[i].z * rs, x[i].w * rs);
            if (p.w) {
                const float4 k = load4<VEC, S>(p.w, c, n);
                v = make_float4(v.x * k.x, v.y * k.y, v.z * k.z, v.w * k.w);
            }
            if constexpr (!QUANT) {
                store4<VEC, S>(p.Y + r * p.ldy, c, n, v);
            } else {
                float top = max4(v);  // (fmaxf drops a NaN: it stays one, and the others keep a scale)
#pragma unroll
                for (int o = S / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const int e = scale_exponent(top);
                store_bytes<VEC, S>(p.Q + r * p.ldq, c, n, e4m3x4(v, power_of_two(-e)));
                const int64_t group = T <= 32 ? i : t / 32 + (int64_t)(T / 32) * i;
                if (t % S == 0 && group * kGroup < n) p.scales[r * p.ldscales + group] = power_of_two(e);
            }
        }
        if (t == 0 && real && p.rstd) p.rstd[r] = rs;
    }
}

struct RmsBwd {
    int64_t M, N;
    const float* dY;
    int64_t lddy;
    const float* S;
    int64_t lds;
    const float *w, *rstd;
    const float* add;  // may be null
    int64_t ldadd;
    float* dX;         // may be null
    int64_t lddx;
    float* partial;    // sums of dw over the rows of each block, or null
};

template <int T, int NV, bool VEC>
__global__ void __launch_bounds__(kBlockThreads<T>) rms_bwd_regs_kernel(const __grid_constant__ RmsBwd p) {
    constexpr int G = kBlockRows<T>, S = kStride<T>;
    const int t = threadIdx.x % T, g = threadIdx.x / T;
    const float inv_n = 1.0f / (float)p.N;
    const int64_t step = (int64_t)gridDim.x * G;
    int flip = 0;
    float4 dw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) dw[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t first = blockIdx.x * (int64_t)G; first < p.M; first += step) {
        const int64_t r = first + g;
        const bool real = r < p.M;
        const int64_t n = real ? p.N : 0;
        float4 x[NV], y[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = load4<VEC, S>(p.S + r * p.lds, first_col<T, VEC>(t, i), n);
            y[i] = load4<VEC, S>(p.dY + r * p.lddy, first_col<T, VEC>(t, i), n);
        }
        const float rs = real ? p.rstd[r] : 0.f;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = make_float4(x[i].x * rs, x[i].y * rs, x[i].z * rs, x[i].w * rs);
            dw[i] = make_float4(fmaf(y[i].x, x[i].x, dw[i].x), fmaf(y[i].y, x[i].y, dw[i].y),
                                fmaf(y[i].z, x[i].z, dw[i].z), fmaf(y[i].w, x[i].w, dw[i].w));
            if (p.w) {
                const float4 k = load4<VEC, S>(p.w, first_col<T, VEC>(t, i), p.N);
                y[i] = make_float4(y[i].x * k.x, y[i].y * k.y, y[i].z * k.z, y[i].w * k.w);
            }
            s += fmaf(y[i].x, x[i].x, y[i].y * x[i].y) + fmaf(y[i].z, x[i].z, y[i].w * x[i].w);
        }
        if (p.dX) {
            const float m = row_sum2<T>(s, 0.f, flip).x * inv_n;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = first_col<T, VEC>(t, i);
                float4 v = make_float4(rs * (y[i].x - x[i].x * m), rs * (y[i].y - x[i].y * m), rs * (y[i].z - x[i].z * m),
                                       rs * (y[i].w - x[i].w * m));
                if (p.add) {
                    const float4 a = load4<VEC, S>(p.add + r * p.ldadd, c, n);
                    v = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
                }
                store4<VEC, S>(p.dX + r * p.lddx, c, n, v);
            }
        }
    }
    if (!p.partial) return;
    if (threadIdx.x == 0) griddep_launch_dependents();  // the partial sums' kernel: its launch, not its reads
    float* out = p.partial + (int64_t)blockIdx.x * p.N;
    if constexpr (T <= 32) {
        // the sums of the block's G groups of threads, added in order
        __shared__ float4 part[G][T * NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) part[g][T * i + t] = dw[i];
        __syncthreads();
        for (int q = threadIdx.x; q < T * NV; q += 256) {
            float4 v = part[0][q];
            for (int i = 1; i < G; ++i) {
                const float4 k = part[i][q];
                v = make_float4(v.x + k.x, v.y + k.y, v.z + k.z, v.w + k.w);
            }
            store4<VEC, S>(out, first_col<T, VEC>(q % T, q / T), p.N, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) store4<VEC, S>(out, first_col<T, VEC>(t, i), p.N, dw[i]);
    }
}

constexpr int64_t kMaxRegsWidth = 16384;

// f(T, NV) for the width.
template <bool BWD, class F> void for_width(int64_t N, F f) {
    auto of = [&](auto T, auto NV) { f(T, NV); };
    using std::integral_constant;
#define EMU_WIDTH(T, NV) of(integral_constant<int, T>{}, integral_constant<int, NV>{})
    if (N <= 16) EMU_WIDTH(4, 1);
    else if (N <= 32) EMU_WIDTH(8, 1);
    else if (N <= 64) EMU_WIDTH(16, 1);
    else if (N <= 128) EMU_WIDTH(32, 1);
    else if (N <= 256) EMU_WIDTH(32, 2);
    else if (N <= 512) EMU_WIDTH(32, 4);
    else if (N <= 1024) EMU_WIDTH(128, 2);
    else if (N <= 2048) EMU_WIDTH(BWD ? 128 : 256, BWD ? 4 : 2);
    else if (N <= 4096) EMU_WIDTH(256, 4);
    else if (N <= 8192) EMU_WIDTH(512, 4);
    else EMU_WIDTH(512, 8);
#undef EMU_WIDTH
}

// ------------------------------------------------------------- wide rows ---
// Two passes over a row: the second finds it in L2.  A thread adds its squares, four at
// a time, in two words as well: it has more of them than of a row in registers.
// 2048 x 20000 119 us, x 32768 195 (2750 GB/s counted once; 2048 x 16384 in registers
// 47.5, 5650 GB/s): word by word, at eight blocks an SM (40 registers: 122 and 200).
template <bool QUANT> __global__ void __launch_bounds__(kRowThreads, 8) rms_fwd_kernel(const __grid_constant__ RmsFwd p) {
    const float inv_n = 1.0f / (float)p.N;
    int flip = 0;
    for (int64_t r = blockIdx.x; r < p.M; r += gridDim.x) {
        const float *x = p.X + r * p.ldx, *q = p.R ? p.R + r * p.ldr : nullptr;
        float s = 0.f, low = 0.f;
        for (int64_t c = threadIdx.x; c < p.N; c += 4 * kRowThreads) {
            float4 v = load4<false, kRowThreads>(x, c, p.N);
            if (q) {
                const float4 k = load4<false, kRowThreads>(q, c, p.N);
                v = make_float4(v.x + k.x, v.y + k.y, v.z + k.z, v.w + k.w);
            }
            if (p.S) store4<false, kRowThreads>(p.S + r * p.lds, c, p.N, v);
            const float2 sum = two_sum(s, fmaf(v.x, v.x, v.y * v.y) + fmaf(v.z, v.z, v.w * v.w));
            s = sum.x;
            low += sum.y;
        }
        const float rs = rstd_of(row_sum_exact<kRowThreads>(s, low, flip), inv_n, p.eps);
        if (threadIdx.x == 0 && p.rstd) p.rstd[r] = rs;
        auto value = [&](int64_t c) {
            float v = (q ? x[c] + q[c] : x[c]) * rs;
            return p.w ? v * p.w[c] : v;
        };
        if constexpr (!QUANT) {
            for (int64_t c = threadIdx.x; c < p.N; c += kRowThreads) p.Y[r * p.ldy + c] = value(c);
        } else {
            const int lane = threadIdx.x & 31;
            for (int64_t g = threadIdx.x >> 5; g * kGroup < p.N; g += kRowThreads / 32) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                const int64_t c = g * kGroup + lane;
                if (c < p.N) v.x = value(c);
                if (c + 32 < p.N) v.y = value(c + 32);
                if (c + 64 < p.N) v.z = value(c + 64);
                if (c + 96 < p.N) v.w = value(c + 96);
                float top = max4(v);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const int e = scale_exponent(top);
                store_bytes<false, 32>(p.Q + r * p.ldq, c, p.N, e4m3x4(v, power_of_two(-e)));
                if (lane == 0) p.scales[r * p.ldscales + g] = power_of_two(e);
            }
        }
    }
}

__global__ void __launch_bounds__(kRowThreads) rms_bwd_dx_kernel(const __grid_constant__ RmsBwd p) {
    for (int64_t r = blockIdx.x; r < p.M; r += gridDim.x) {
        const float *x = p.S + r * p.lds, *dy = p.dY + r * p.lddy;
        const float rs = p.rstd[r];
        float s = 0.f;
        for (int64_t c = threadIdx.x; c < p.N; c += kRowThreads) s = fmaf(p.w ? dy[c] * p.w[c] : dy[c], x[c] * rs, s);
        const float m = block_sum2(s, 0.f).x / (float)p.N;
        for (int64_t c = threadIdx.x; c < p.N; c += kRowThreads) {
            const float g = p.w ? dy[c] * p.w[c] : dy[c];
            float v = rs * (g - x[c] * rs * m);
            if (p.add) v += p.add[r * p.ldadd + c];
            p.dX[r * p.lddx + c] = v;
        }
    }
}

// partial[blockIdx.y][c]: dw over this block's rows
__global__ void __launch_bounds__(256) rms_bwd_weight_kernel(const __grid_constant__ RmsBwd p, int64_t rows_per) {
    const int64_t c = blockIdx.x * 256ll + threadIdx.x;
    if (c >= p.N) return;
    const int64_t r0 = blockIdx.y * rows_per, r1 = r0 + rows_per < p.M ? r0 + rows_per : p.M;
    float dw = 0.f;
    for (int64_t r = r0; r < r1; ++r) dw = fmaf(p.dY[r * p.lddy + c], p.S[r * p.lds + c] * p.rstd[r], dw);
    p.partial[(int64_t)blockIdx.y * p.N + c] = dw;
}

template <bool QUANT> cudaError_t launch_fwd(const RmsFwd& p, int sm_count, cudaStream_t s) {
    cudaGetLastError();
    if (p.N > kMaxRegsWidth) {
        const int64_t grid = p.M < sm_count * 8 ? p.M : sm_count * 8;
        rms_fwd_kernel<QUANT><<<(unsigned)grid, kRowThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    const bool vec = (p.N & 3) == 0 && vec4_ok(p.X, p.ldx) && vec4_ok(p.R, p.R ? p.ldr : 0) && vec4_ok(p.w, 0) &&
                     vec4_ok(p.S, p.S ? p.lds : 0) &&
                     (QUANT ? (reinterpret_cast<uintptr_t>(p.Q) & 3) == 0 && (p.ldq & 3) == 0 : vec4_ok(p.Y, p.ldy));
    for_width<false>(p.N, [&](auto T, auto NV) {
        constexpr int t = decltype(T)::value, nv = decltype(NV)::value;
        auto launch = [&](auto VEC) {
            constexpr auto kernel = rms_fwd_regs_kernel<t, nv, decltype(VEC)::value, QUANT>;
            static const int per_sm = resident_blocks(kernel, kBlockThreads<t>);
            kernel<<<even_grid(p.M, kBlockRows<t>, (int64_t)sm_count * per_sm), kBlockThreads<t>, 0, s>>>(p);
        };
        if (vec) launch(std::true_type{}); else launch(std::false_type{});
    });
    return cudaGetLastError();
}

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" {

emu_status_t emu_rms_norm_fwd(int64_t M, int64_t N, const float* X, int64_t ldx, const float* residual, int64_t ldr,
                              const float* weight, float eps, float* Y, int64_t ldy, float* S, int64_t lds, float* rstd,
                              emu_stream_t stream) {
    if (M < 0 || N < 0 || !(eps >= 0.0f)) return EMU_STATUS_INVALID_VALUE;
    if (N > INT32_MAX - 256) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0 || N == 0) return EMU_STATUS_SUCCESS;
    if (!X || !Y || ldx < N || ldy < N || (residual && ldr < N) || (S && lds < N)) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev;
    const emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    const RmsFwd p{M, N, X, ldx, residual, ldr, weight, eps, S, lds, rstd, Y, ldy, nullptr, 0, nullptr, 0};
    return launch_fwd<false>(p, dev.sm_count, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED;
}

emu_status_t emu_rms_norm_quant(int64_t M, int64_t N, const float* X, int64_t ldx, const float* residual, int64_t ldr,
                                const float* weight, float eps, uint8_t* Q, int64_t ldq, float* scales, int64_t ldscales,
                                float* S, int64_t lds, emu_stream_t stream) {
    if (M < 0 || N < 0 || !(eps >= 0.0f)) return EMU_STATUS_INVALID_VALUE;
    if (N > INT32_MAX - 256) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0 || N == 0) return EMU_STATUS_SUCCESS;
    if (!X || !Q || !scales || ldx < N || ldq < N || ldscales < (N + kGroup - 1) / kGroup || (residual && ldr < N) ||
        (S && lds < N))
        return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev;
    const emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    const RmsFwd p{M, N, X, ldx, residual, ldr, weight, eps, S, lds, nullptr, nullptr, 0, Q, ldq, scales, ldscales};
    return launch_fwd<true>(p, dev.sm_count, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED;
}

emu_status_t emu_rms_norm_bwd(int64_t M, int64_t N, const float* dY, int64_t lddy, const float* S, int64_t lds,
                              const float* weight, const float* rstd, const float* add, int64_t ldadd, float* dX,
                              int64_t lddx, float* dweight, emu_stream_t stream) {
    if (M < 0 || N < 0) return EMU_STATUS_INVALID_VALUE;
    if (N > INT32_MAX - 256) return EMU_STATUS_NOT_SUPPORTED;
    if (N == 0) return EMU_STATUS_SUCCESS;
    if (M > 0 && (!dY || !S || !rstd || lddy < N || lds < N || (dX && lddx < N) || (add && ldadd < N)))
        return EMU_STATUS_INVALID_VALUE;
    if (add && !dX) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev;
    emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    if (M == 0) {  // an empty sum
        if (dweight && cudaMemsetAsync(dweight, 0, N * sizeof(float), s) != cudaSuccess) {
            cudaGetLastError();
            return EMU_STATUS_LAUNCH_FAILED;
        }
        return EMU_STATUS_SUCCESS;
    }
    if (!dX && !dweight) return EMU_STATUS_SUCCESS;
    RmsBwd p{M, N, dY, lddy, S, lds, weight, rstd, add, ldadd, dX, lddx, nullptr};
    cudaError_t e = cudaSuccess;
    int64_t chunks = 0;
    if (N <= kMaxRegsWidth) {
        const bool vec = (N & 3) == 0 && vec4_ok(dY, lddy) && vec4_ok(S, lds) && vec4_ok(weight, 0) &&
                         vec4_ok(add, add ? ldadd : 0) && vec4_ok(dX, dX ? lddx : 0);
        for_width<true>(N, [&](auto T, auto NV) {
            constexpr int t = decltype(T)::value, nv = decltype(NV)::value;
            auto launch = [&](auto VEC) {
                constexpr auto kernel = rms_bwd_regs_kernel<t, nv, decltype(VEC)::value>;
                static const int per_sm = resident_blocks(kernel, kBlockThreads<t>);
                const unsigned grid = even_grid(M, kBlockRows<t>, (int64_t)dev.sm_count * per_sm);
                chunks = grid;
                if (dweight) st = reduce_scratch(dev.id, s, (size_t)grid * N, &p.partial);
                if (st != EMU_STATUS_SUCCESS) return;
                cudaGetLastError();
                kernel<<<grid, kBlockThreads<t>, 0, s>>>(p);
                e = cudaGetLastError();
            };
            if (vec) launch(std::true_type{}); else launch(std::false_type{});
        });
        if (st != EMU_STATUS_SUCCESS) return st;
    } else {
        const int64_t col_blocks = (N + 255) / 256;
        chunks = (dev.sm_count * 8 + col_blocks - 1) / col_blocks;
        if (chunks > (M + 31) / 32) chunks = (M + 31) / 32;
        const int64_t rows_per = (M + chunks - 1) / chunks;
        chunks = (M + rows_per - 1) / rows_per;
        if (dweight) st = reduce_scratch(dev.id, s, (size_t)chunks * N, &p.partial);
        if (st != EMU_STATUS_SUCCESS) return st;
        cudaGetLastError();
        const int64_t grid = M < dev.sm_count * 8 ? M : dev.sm_count * 8;
        if (dX) rms_bwd_dx_kernel<<<(unsigned)grid, kRowThreads, 0, s>>>(p);
        if (dweight) rms_bwd_weight_kernel<<<dim3((unsigned)col_blocks, (unsigned)chunks), 256, 0, s>>>(p, rows_per);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return EMU_STATUS_LAUNCH_FAILED;
    const Partials sums{p.partial, (int)chunks, N, N, dweight, nullptr};
    return !dweight || launch_sum_partials(&sums, 1, s) == cudaSuccess ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED;
}

}  // extern "C"
