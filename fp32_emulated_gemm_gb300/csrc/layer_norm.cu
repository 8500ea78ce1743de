// layer_norm.cu -- layer normalisation over the rows of an FP32 matrix,
// forward and backward, with the reductions of the weight's and the bias's
// gradients.
//
// Row x of width N: mu = sum x / N, r = 1 / sqrt(sum (x - mu)^2 / N + eps),
// xh = (x - mu) r, y = xh w + b.  Backward, with g = dy w:
//   dx = r (g - mean(g) - xh mean(g xh)) (+ add),
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
#include <cuda_runtime.h>

#include "internal.h"
#include "row_ops.cuh"

namespace emu {
namespace {

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

// One block per row, three passes over it.
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

__global__ void __launch_bounds__(1024) sum_partials_kernel(const float* partial, int P, int64_t C, int64_t split,
                                                            float* out0, float* out1) {
    __shared__ float part[32][33];
    const int64_t c = blockIdx.x * 32ll + threadIdx.x;
    float s = 0.f;
    if (c < C)
        for (int p = threadIdx.y; p < P; p += 32) s += partial[(int64_t)p * C + c];
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < C) {
        float t = part[0][threadIdx.x];
        for (int i = 1; i < 32; ++i) t += part[i][threadIdx.x];
        if (c < split) { if (out0) out0[c] = t; }
        else if (out1) out1[c - split] = t;
    }
}
cudaError_t launch_sum_partials(const float* partial, int P, int64_t C, int64_t split, float* out0, float* out1,
                                cudaStream_t stream) {
    cudaGetLastError();
    sum_partials_kernel<<<(unsigned)((C + 31) / 32), dim3(32, 32), 0, stream>>>(partial, P, C, split, out0, out1);
    return cudaGetLastError();
}

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
    cudaGetLastError();
    const int64_t grid = M < dev.sm_count * 8 ? M : dev.sm_count * 8;
    ln_fwd_kernel<<<(unsigned)grid, kRowThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        M, N, X, ldx, weight, bias, eps, Y, ldy, mean, rstd);
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
    const bool params = dweight || dbias;
    if (M == 0) {  // empty sums
        if ((dweight && cudaMemsetAsync(dweight, 0, N * sizeof(float), s) != cudaSuccess) ||
            (dbias && cudaMemsetAsync(dbias, 0, N * sizeof(float), s) != cudaSuccess)) {
            cudaGetLastError();
            return EMU_STATUS_LAUNCH_FAILED;
        }
        return EMU_STATUS_SUCCESS;
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
    if (params && launch_sum_partials(partial, (int)chunks, 2 * N, N, dweight, dbias, s) != cudaSuccess)
        return EMU_STATUS_LAUNCH_FAILED;
    return EMU_STATUS_SUCCESS;
}

}  // extern "C"
