// layer_norm.cu -- layer normalisation over the rows of an FP32 matrix,
// forward and backward, with the reductions of the weight's and the bias's
// gradients.
//
// Row x of width N: mu = sum x / N, r = 1 / sqrt(sum (x - mu)^2 / N + eps),
// xh = (x - mu) r, y = xh w + b.  Backward, with g = dy w:
//   dx = r (g - mean(g) - xh mean(g xh)) (+ add),
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"
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

template <int T, int NV, bool VEC>
__global__ void __launch_bounds__(kBlockThreads<T>)
ln_fwd_regs_kernel(int64_t M, int64_t N, const float* __restrict__ X, int64_t ldx, const float* __restrict__ w,
                   const float* __restrict__ b, float eps, float* __restrict__ Y, int64_t ldy, float* mean, float* rstd) {
    constexpr int G = kBlockRows<T>;
    const int t = threadIdx.x % T, g = threadIdx.x / T;
    const float inv_n = 1.0f / (float)N;
    const int64_t step = (int64_t)gridDim.x * G;
    int flip = 0;
    // (the loop is the same for all threads of a block: shuffles and barriers)
    for (int64_t first = blockIdx.x * (int64_t)G; first < M; first += step) {
        const int64_t r = first + g;
        const bool real = r < M;
        float4 x[NV];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = load4<VEC, T>(X + r * ldx, col_of<T, VEC>(t, i), real ? N : 0);
#pragma unroll
        for (int i = 0; i < NV; ++i) s += (x[i].x + x[i].y) + (x[i].z + x[i].w);
        const float mu = row_sum2<T>(s, 0.f, flip).x * inv_n;
        // the squared deviations from the mean just found, not E x^2 - mu^2:
        // no cancellation when the mean is large
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = col_of<T, VEC>(t, i);
            x[i] = make_float4(x[i].x - mu, x[i].y - mu, x[i].z - mu, x[i].w - mu);
            if (inside<T, VEC>(c, 0, N)) q = fmaf(x[i].x, x[i].x, q);
            if (inside<T, VEC>(c, 1, N)) q = fmaf(x[i].y, x[i].y, q);
            if (inside<T, VEC>(c, 2, N)) q = fmaf(x[i].z, x[i].z, q);
            if (inside<T, VEC>(c, 3, N)) q = fmaf(x[i].w, x[i].w, q);
        }
        const float rs = 1.0f / sqrtf(fmaf(row_sum2<T>(q, 0.f, flip).x, inv_n, eps));
        if (!real) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = col_of<T, VEC>(t, i);
            float4 v = make_float4(x[i].x * rs, x[i].y * rs, x[i].z * rs, x[i].w * rs);
            if (w) {
                const float4 k = load4<VEC, T>(w, c, N);
                v = make_float4(v.x * k.x, v.y * k.y, v.z * k.z, v.w * k.w);
            }
            if (b) {
                const float4 k = load4<VEC, T>(b, c, N);
                v = make_float4(v.x + k.x, v.y + k.y, v.z + k.z, v.w + k.w);
            }
            store4<VEC, T>(Y + r * ldy, c, N, v);
        }
        if (t == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

// dX and, over the rows this block takes, the sums of dw and db, which stay in
// registers until the end and go to partial[blockIdx.x][0 and 1][column].
template <int T, int NV, bool VEC>
__global__ void __launch_bounds__(kBlockThreads<T>, T <= 32 && NV <= 2 ? 4 : 1)
ln_bwd_regs_kernel(int64_t M, int64_t N, const float* __restrict__ dY, int64_t lddy, const float* __restrict__ X,
                   int64_t ldx, const float* __restrict__ w, const float* __restrict__ mean,
                   const float* __restrict__ rstd, const float* __restrict__ add, int64_t ldadd, float* __restrict__ dX,
                   int64_t lddx, float* __restrict__ partial) {
    constexpr int G = kBlockRows<T>;
    const int t = threadIdx.x % T, g = threadIdx.x / T;
    const float inv_n = 1.0f / (float)N;
    const int64_t step = (int64_t)gridDim.x * G;
    int flip = 0;
    float4 dw[NV], db[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) dw[i] = db[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t first = blockIdx.x * (int64_t)G; first < M; first += step) {
        const int64_t r = first + g;
        const bool real = r < M;
        float4 x[NV], y[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = load4<VEC, T>(X + r * ldx, col_of<T, VEC>(t, i), real ? N : 0);
            y[i] = load4<VEC, T>(dY + r * lddy, col_of<T, VEC>(t, i), real ? N : 0);
        }
        const float mu = real ? mean[r] : 0.f, rs = real ? rstd[r] : 0.f;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = make_float4((x[i].x - mu) * rs, (x[i].y - mu) * rs, (x[i].z - mu) * rs, (x[i].w - mu) * rs);
            dw[i] = make_float4(fmaf(y[i].x, x[i].x, dw[i].x), fmaf(y[i].y, x[i].y, dw[i].y),
                                fmaf(y[i].z, x[i].z, dw[i].z), fmaf(y[i].w, x[i].w, dw[i].w));
            db[i] = make_float4(db[i].x + y[i].x, db[i].y + y[i].y, db[i].z + y[i].z, db[i].w + y[i].w);
            if (w) {
                const float4 k = load4<VEC, T>(w, col_of<T, VEC>(t, i), N);
                y[i] = make_float4(y[i].x * k.x, y[i].y * k.y, y[i].z * k.z, y[i].w * k.w);
            }
            // (outside the row dY is zero, whatever xh is)
            s1 += (y[i].x + y[i].y) + (y[i].z + y[i].w);
            s2 += fmaf(y[i].x, x[i].x, y[i].y * x[i].y) + fmaf(y[i].z, x[i].z, y[i].w * x[i].w);
        }
        if (dX) {
            const float2 m = row_sum2<T>(s1, s2, flip);
            const float m1 = m.x * inv_n, m2 = m.y * inv_n;
            if (real) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int64_t c = col_of<T, VEC>(t, i);
                    float4 v = make_float4(rs * (y[i].x - m1 - x[i].x * m2), rs * (y[i].y - m1 - x[i].y * m2),
                                           rs * (y[i].z - m1 - x[i].z * m2), rs * (y[i].w - m1 - x[i].w * m2));
                    if (add) {
                        const float4 a = load4<VEC, T>(add + r * ldadd, c, N);
                        v = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
                    }
                    store4<VEC, T>(dX + r * lddx, c, N, v);
                }
            }
        }
    }
    if (!partial) return;
    if (threadIdx.x == 0) griddep_launch_dependents();  // the partial sums' kernel: its launch, not its reads
    float* out = partial + (int64_t)blockIdx.x * 2 * N;
    if constexpr (T <= 32) {
        // the sums of the block's G groups of threads, added in order
        __shared__ float4 part[2][G][T * NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            part[0][g][T * i + t] = dw[i];
            part[1][g][T * i + t] = db[i];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * T * NV; e += 256) {
            const int which = e / (T * NV), q = e % (T * NV);
            float4 v = part[which][0][q];
            for (int i = 1; i < G; ++i) {
                const float4 k = part[which][i][q];
                v = make_float4(v.x + k.x, v.y + k.y, v.z + k.z, v.w + k.w);
            }
            store4<VEC, T>(out + which * N, col_of<T, VEC>(q % T, q / T), N, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            store4<VEC, T>(out, col_of<T, VEC>(t, i), N, dw[i]);
            store4<VEC, T>(out + N, col_of<T, VEC>(t, i), N, db[i]);
        }
    }
}

constexpr int64_t kMaxRegsWidth = 16384;

// f(T, NV) for the width.  Measured fractions of the copy rate, forward and
// backward, at 0.4 GB a matrix: N = 16 0.88 and 0.85, 32 0.88 and 0.86, 61
// (unaligned rows) 0.73 and 0.79, 128 0.87 and 0.94, 256 0.93 and 0.93, 512 0.94
// and 0.94, 1024 0.95 and 0.95, 2048 0.96 and 0.93 (backward with 256 threads
// of 2: 0.87), 4096 0.90 and 0.88 (512 threads of 2: 0.83 and 0.60; 128 of 8:
// 0.85 and 0.85), 8192 0.94 and 0.77 (256 of 8: 0.85 and 0.77), 16384 0.84 and
// 0.62 (1024 of 4: 0.62 and 0.58; the backward kernel holds x, dY, dw and db in
// eight float4 each, which are all of its 128 registers, and spills 184 to 208
// bytes a thread).  Copying the rows after next to shared
// memory meanwhile was slower at every width up to 4096.
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

// How many blocks of the forward kernel an SM takes (at most `resident`) when X
// is larger than L2: with every block resident the reads and writes in flight
// get in each other's way.  About 43 KB of rows per SM were fastest up to a
// width of 1024 (fractions of the copy rate, all resident / 43 KB: 256 0.83 /
// 0.93, 512 0.88 / 0.94, 1024 0.87 / 0.95; up to 128 columns all are less),
// 64 KB for 2048 and 4096 (0.86 / 0.90), 96 KB above.  Smaller matrices, and
// the backward kernel, which holds more registers, want all of them.
int64_t forward_blocks(int64_t M, int64_t N, int rows, int resident) {
    if (M * N * (int64_t)sizeof(float) < (int64_t(100) << 20)) return resident;
    const int64_t target = (N <= 1024 ? 43 : N <= 4096 ? 64 : 96) << 10, block = rows * N * (int64_t)sizeof(float);
    const int64_t n = (target + block / 2) / block;
    return n < 1 ? 1 : n < resident ? n : resident;
}

// Blocks that take the rows in turns of equal length: at most `resident`.
unsigned even_grid(int64_t M, int rows, int64_t resident) {
    const int64_t groups = (M + rows - 1) / rows, turns = (groups + resident - 1) / resident;
    return (unsigned)((groups + turns - 1) / turns);
}

// ------------------------------------------------------------- wide rows ---
// Rows wider than the registers hold: a block a row, several passes over it.
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

__global__ void __launch_bounds__(kRowThreads)
ln_fwd_kernel(int64_t M, int64_t N, const float* X, int64_t ldx, const float* w, const float* b, float eps, float* Y,
              int64_t ldy, float* mean, float* rstd) {
    for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
        const float* x = X + r * ldx;
        float s = 0.f;
        for (int64_t c = threadIdx.x; c < N; c += kRowThreads) s += x[c];
        const float mu = block_sum2(s, 0.f).x / (float)N;
        float q = 0.f;
        for (int64_t c = threadIdx.x; c < N; c += kRowThreads) { const float d = x[c] - mu; q = fmaf(d, d, q); }
        const float rs = 1.0f / sqrtf(block_sum2(q, 0.f).x / (float)N + eps);
        float* y = Y + r * ldy;
        for (int64_t c = threadIdx.x; c < N; c += kRowThreads) {
            float v = (x[c] - mu) * rs;
            if (w) v *= w[c];
            if (b) v += b[c];
            y[c] = v;
        }
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

__global__ void __launch_bounds__(kRowThreads)
ln_bwd_dx_kernel(int64_t M, int64_t N, const float* dY, int64_t lddy, const float* X, int64_t ldx, const float* w,
                 const float* mean, const float* rstd, const float* add, int64_t ldadd, float* dX, int64_t lddx) {
    for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
        const float *x = X + r * ldx, *dy = dY + r * lddy;
        const float mu = mean[r], rs = rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int64_t c = threadIdx.x; c < N; c += kRowThreads) {
            const float g = w ? dy[c] * w[c] : dy[c];
            s1 += g;
            s2 = fmaf(g, (x[c] - mu) * rs, s2);
        }
        const float2 t = block_sum2(s1, s2);
        const float m1 = t.x / (float)N, m2 = t.y / (float)N;
        for (int64_t c = threadIdx.x; c < N; c += kRowThreads) {
            const float g = w ? dy[c] * w[c] : dy[c], xh = (x[c] - mu) * rs;
            float v = rs * (g - m1 - xh * m2);
            if (add) v += add[r * ldadd + c];
            dX[r * lddx + c] = v;
        }
    }
}

// partial[blockIdx.y][0][c], [1][c]: dw and db over this block's rows
__global__ void __launch_bounds__(256)
ln_bwd_params_kernel(int64_t M, int64_t N, int64_t rows_per, const float* dY, int64_t lddy, const float* X, int64_t ldx,
                     const float* mean, const float* rstd, float* partial) {
    const int64_t c = blockIdx.x * 256ll + threadIdx.x;
    if (c >= N) return;
    const int64_t r0 = blockIdx.y * rows_per, r1 = r0 + rows_per < M ? r0 + rows_per : M;
    float dw = 0.f, db = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = dY[r * lddy + c];
        dw = fmaf(dy, (X[r * ldx + c] - mean[r]) * rstd[r], dw);
        db += dy;
    }
    partial[(int64_t)blockIdx.y * 2 * N + c] = dw;
    partial[(int64_t)blockIdx.y * 2 * N + N + c] = db;
}

}  // namespace

}  // namespace emu

using namespace emu;

extern "C" {

emu_status_t emu_layer_norm_fwd(int64_t M, int64_t N, const float* X, int64_t ldx, const float* weight,
                                const float* bias, float eps, float* Y, int64_t ldy, float* mean, float* rstd,
                                emu_stream_t stream) {
    if (M < 0 || N < 0 || !(eps >= 0.0f)) return EMU_STATUS_INVALID_VALUE;
    if (N > INT32_MAX - 256) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0 || N == 0) return EMU_STATUS_SUCCESS;
    if (!X || !Y || ldx < N || ldy < N) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev;
    const emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaGetLastError();
    if (N <= kMaxRegsWidth) {
        const bool vec = (N & 3) == 0 && vec4_ok(X, ldx) && vec4_ok(Y, ldy) && vec4_ok(weight, 0) && vec4_ok(bias, 0);
        for_width<false>(N, [&](auto T, auto NV) {
            constexpr int t = decltype(T)::value, nv = decltype(NV)::value;
            auto launch = [&](auto VEC) {
                constexpr auto kernel = ln_fwd_regs_kernel<t, nv, decltype(VEC)::value>;
                static const int per_sm = resident_blocks(kernel, kBlockThreads<t>);
                const unsigned grid =
                    even_grid(M, kBlockRows<t>, dev.sm_count * forward_blocks(M, N, kBlockRows<t>, per_sm));
                kernel<<<grid, kBlockThreads<t>, 0, s>>>(M, N, X, ldx, weight, bias, eps, Y, ldy, mean, rstd);
            };
            if (vec) launch(std::true_type{}); else launch(std::false_type{});
        });
    } else {
        const int64_t grid = M < dev.sm_count * 8 ? M : dev.sm_count * 8;
        ln_fwd_kernel<<<(unsigned)grid, kRowThreads, 0, s>>>(M, N, X, ldx, weight, bias, eps, Y, ldy, mean, rstd);
    }
    return cudaGetLastError() == cudaSuccess ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED;
}

emu_status_t emu_layer_norm_bwd(int64_t M, int64_t N, const float* dY, int64_t lddy, const float* X, int64_t ldx,
                                const float* weight, const float* mean, const float* rstd, const float* add,
                                int64_t ldadd, float* dX, int64_t lddx, float* dweight, float* dbias,
                                emu_stream_t stream) {
    if (M < 0 || N < 0) return EMU_STATUS_INVALID_VALUE;
    if (N > INT32_MAX - 256) return EMU_STATUS_NOT_SUPPORTED;
    if (N == 0) return EMU_STATUS_SUCCESS;
    if (M > 0 && (!dY || !X || !mean || !rstd || lddy < N || ldx < N || (dX && lddx < N) || (add && ldadd < N)))
        return EMU_STATUS_INVALID_VALUE;
    if (add && !dX) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev;
    emu_status_t st = current_device(&dev);
    if (st != EMU_STATUS_SUCCESS) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    const bool params = dweight || dbias;
    if (M == 0) {  // empty sums
        if ((dweight && cudaMemsetAsync(dweight, 0, N * sizeof(float), s) != cudaSuccess) ||
            (dbias && cudaMemsetAsync(dbias, 0, N * sizeof(float), s) != cudaSuccess)) {
            cudaGetLastError();
            return EMU_STATUS_LAUNCH_FAILED;
        }
        return EMU_STATUS_SUCCESS;
    }
    if (N <= kMaxRegsWidth) {
        const bool vec = (N & 3) == 0 && vec4_ok(dY, lddy) && vec4_ok(X, ldx) && vec4_ok(weight, 0) &&
                         vec4_ok(add, add ? ldadd : 0) && vec4_ok(dX, dX ? lddx : 0);
        cudaError_t e = cudaSuccess;
        for_width<true>(N, [&](auto T, auto NV) {
            constexpr int t = decltype(T)::value, nv = decltype(NV)::value;
            auto launch = [&](auto VEC) {
                constexpr auto kernel = ln_bwd_regs_kernel<t, nv, decltype(VEC)::value>;
                static const int per_sm = resident_blocks(kernel, kBlockThreads<t>);
                const unsigned grid = even_grid(M, kBlockRows<t>, (int64_t)dev.sm_count * per_sm);
                float* partial = nullptr;
                if (params) st = reduce_scratch(dev.id, s, (size_t)grid * 2 * N, &partial);
                if (st != EMU_STATUS_SUCCESS) return;
                cudaGetLastError();
                kernel<<<grid, kBlockThreads<t>, 0, s>>>(M, N, dY, lddy, X, ldx, weight, mean, rstd, add, ldadd, dX, lddx,
                                                         partial);
                e = cudaGetLastError();
                const Partials sums{partial, (int)grid, 2 * N, N, dweight, dbias};
                if (e == cudaSuccess && params) e = launch_sum_partials(&sums, 1, s);
            };
            if (vec) launch(std::true_type{}); else launch(std::false_type{});
        });
        if (st != EMU_STATUS_SUCCESS) return st;
        return e == cudaSuccess ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED;
    }
    const int64_t col_blocks = (N + 255) / 256;
    int64_t chunks = (dev.sm_count * 8 + col_blocks - 1) / col_blocks;
    if (chunks > (M + 31) / 32) chunks = (M + 31) / 32;
    const int64_t rows_per = (M + chunks - 1) / chunks;
    chunks = (M + rows_per - 1) / rows_per;
    float* partial = nullptr;
    if (params) {
        st = reduce_scratch(dev.id, s, (size_t)chunks * 2 * N, &partial);
        if (st != EMU_STATUS_SUCCESS) return st;
    }
    cudaGetLastError();
    if (dX) {
        const int64_t grid = M < dev.sm_count * 8 ? M : dev.sm_count * 8;
        ln_bwd_dx_kernel<<<(unsigned)grid, kRowThreads, 0, s>>>(M, N, dY, lddy, X, ldx, weight, mean, rstd, add, ldadd,
                                                                dX, lddx);
    }
    if (params)
        ln_bwd_params_kernel<<<dim3((unsigned)col_blocks, (unsigned)chunks), 256, 0, s>>>(M, N, rows_per, dY, lddy, X,
                                                                                          ldx, mean, rstd, partial);
    if (cudaGetLastError() != cudaSuccess) return EMU_STATUS_LAUNCH_FAILED;
    const Partials sums{partial, (int)chunks, 2 * N, N, dweight, dbias};
    if (params && launch_sum_partials(&sums, 1, s) != cudaSuccess) return EMU_STATUS_LAUNCH_FAILED;
    return EMU_STATUS_SUCCESS;
}

}  // extern "C"
