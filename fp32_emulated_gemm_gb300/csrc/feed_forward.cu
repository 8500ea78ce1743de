// feed_forward.cu -- the feed-forward operators around the emulated products:
// a linear layer with bias, activation and residual, and the gated
// feed-forward block, each with its backward pass.
//
//   linear_act: Z = X W^T + b, Y = a(Z) + R
//               dZ = dY a'(Z), dX = dZ W, dW = dZ^T X, db = sum over rows of dZ
//   gated:      [G | U] = Z = X [Wg; Wu]^T + [bg | bu], H = a(G) U
//               dG = dH U a'(G), dU = dH a(G), then as above with dZ = [dG | dU]
//   gated_ffn:  Y = H Wo^T + bo + R;  dH = dY Wo, dWo = dY^T H, dbo = sum of dY
#include <cuda_runtime.h>

#include "activation.cuh"
#include "internal.h"
#include "row_ops.cuh"

namespace emu {
namespace {

// The row-wise kernels: a warp covers 128 columns (a float4 per lane, or four
// words 32 apart where rows are not 16-byte aligned) of one row at a time, the
// eight warps of a block take rows in turn, and a block has one chunk of rows.
constexpr int kWarps = 8, kCols = 128;

struct RowGrid { dim3 grid; int64_t rows_per; int chunks; };
RowGrid row_grid(int64_t M, int64_t N, int sm_count) {
    const int64_t col_blocks = (N + kCols - 1) / kCols;
    int64_t chunks = ((int64_t)sm_count * 8 + col_blocks - 1) / col_blocks;  // eight blocks of 256 threads per SM
    if (chunks > (M + 31) / 32) chunks = (M + 31) / 32;
    const int64_t rows_per = (M + chunks - 1) / chunks;
    chunks = (M + rows_per - 1) / rows_per;
    return {dim3((unsigned)col_blocks, (unsigned)chunks), rows_per, (int)chunks};
}

__device__ __forceinline__ float4 act_value4(int act, const float4& z) {
    return make_float4(act_value(act, z.x), act_value(act, z.y), act_value(act, z.z), act_value(act, z.w));
}

// Y = a(Z) + R, or with GATED H = a(G) U from Z = [G | U] of 2N columns.
template <bool GATED, bool VEC>
__global__ void __launch_bounds__(32 * kWarps)
act_fwd_kernel(int act, int64_t M, int64_t N, int64_t rows_per, const float* Z, int64_t ldz, const float* R, int64_t ldr,
               float* Y, int64_t ldy) {
    constexpr int S = 32;
    const int64_t c = blockIdx.x * (int64_t)kCols + (VEC ? 4 * threadIdx.x : threadIdx.x);
    const int64_t r1 = min(M, (blockIdx.y + 1) * rows_per);
    for (int64_t r = blockIdx.y * rows_per + threadIdx.y; r < r1; r += kWarps) {
        float4 z = load4<VEC, S>(Z + r * ldz, c, N);
        z = act_value4(act, z);
        if constexpr (GATED) {
            const float4 u = load4<VEC, S>(Z + r * ldz + N, c, N);
            z = make_float4(z.x * u.x, z.y * u.y, z.z * u.z, z.w * u.w);
        } else if (R) {
            const float4 q = load4<VEC, S>(R + r * ldr, c, N);
            z = make_float4(z.x + q.x, z.y + q.y, z.z + q.z, z.w + q.w);
        }
        store4<VEC, S>(Y + r * ldy, c, N, z);
    }
}

// dZ = dY a'(Z), or with GATED dG = dH U a'(G), dU = dH a(G) (Z, dZ of 2N
// columns); the sums of this block's rows of dZ go to partial[blockIdx.y].
// Z null: dZ = dY, not written (the sums alone).
template <bool GATED, bool VEC>
__global__ void __launch_bounds__(32 * kWarps)
act_bwd_kernel(int act, int64_t M, int64_t N, int64_t rows_per, const float* dY, int64_t lddy, const float* Z,
               int64_t ldz, float* dZ, int64_t lddz, float* partial) {
    constexpr int S = 32;
    __shared__ float4 sums[GATED ? 2 : 1][kWarps][32];
    const int64_t c = blockIdx.x * (int64_t)kCols + (VEC ? 4 * threadIdx.x : threadIdx.x);
    const int64_t r1 = min(M, (blockIdx.y + 1) * rows_per);
    float4 sg = make_float4(0.f, 0.f, 0.f, 0.f), su = sg;
    for (int64_t r = blockIdx.y * rows_per + threadIdx.y; r < r1; r += kWarps) {
        float4 g = load4<VEC, S>(dY + r * lddy, c, N);
        if (Z) {
            const float4 z = load4<VEC, S>(Z + r * ldz, c, N);
            float4 a, d;
            act_value_grad(act, z.x, a.x, d.x);
            act_value_grad(act, z.y, a.y, d.y);
            act_value_grad(act, z.z, a.z, d.z);
            act_value_grad(act, z.w, a.w, d.w);
            if constexpr (GATED) {
                const float4 u = load4<VEC, S>(Z + r * ldz + N, c, N);
                const float4 du = make_float4(g.x * a.x, g.y * a.y, g.z * a.z, g.w * a.w);
                store4<VEC, S>(dZ + r * lddz + N, c, N, du);
                su = make_float4(su.x + du.x, su.y + du.y, su.z + du.z, su.w + du.w);
                g = make_float4(g.x * u.x, g.y * u.y, g.z * u.z, g.w * u.w);
            }
            g = make_float4(g.x * d.x, g.y * d.y, g.z * d.z, g.w * d.w);
            store4<VEC, S>(dZ + r * lddz, c, N, g);
        }
        sg = make_float4(sg.x + g.x, sg.y + g.y, sg.z + g.z, sg.w + g.w);
    }
    if (!partial) return;
    sums[0][threadIdx.y][threadIdx.x] = sg;
    if constexpr (GATED) sums[1][threadIdx.y][threadIdx.x] = su;
    __syncthreads();
    if (threadIdx.y < (GATED ? 2 : 1)) {
        float4 t = sums[threadIdx.y][0][threadIdx.x];
        for (int i = 1; i < kWarps; ++i) {
            const float4 v = sums[threadIdx.y][i][threadIdx.x];
            t = make_float4(t.x + v.x, t.y + v.y, t.z + v.z, t.w + v.w);
        }
        const int64_t width = (GATED ? 2 : 1) * N;
        float* out = partial + blockIdx.y * width + threadIdx.y * N;
        // (partial rows of odd width: word stores)
        constexpr int W = VEC ? 1 : S;
        if (c < N) out[c] = t.x;
        if (c + W < N) out[c + W] = t.y;
        if (c + 2 * W < N) out[c + 2 * W] = t.z;
        if (c + 3 * W < N) out[c + 3 * W] = t.w;
    }
}

template <bool GATED>
cudaError_t launch_act_fwd(int act, int64_t M, int64_t N, const float* Z, int64_t ldz, const float* R, int64_t ldr,
                           float* Y, int64_t ldy, int sm_count, cudaStream_t s) {
    if (M == 0 || N == 0) return cudaSuccess;
    const RowGrid g = row_grid(M, N, sm_count);
    const bool vec = (N & 3) == 0 && vec4_ok(Z, ldz) && vec4_ok(Y, ldy) && (!R || vec4_ok(R, ldr));
    cudaGetLastError();
    if (vec) act_fwd_kernel<GATED, true><<<g.grid, dim3(32, kWarps), 0, s>>>(act, M, N, g.rows_per, Z, ldz, R, ldr, Y, ldy);
    else act_fwd_kernel<GATED, false><<<g.grid, dim3(32, kWarps), 0, s>>>(act, M, N, g.rows_per, Z, ldz, R, ldr, Y, ldy);
    return cudaGetLastError();
}

// `scratch`: column_sum_floats() floats when dbias is wanted, else null
size_t column_sum_floats(bool gated, int64_t M, int64_t N, int sm_count) {
    return M > 0 && N > 0 ? (size_t)row_grid(M, N, sm_count).chunks * (gated ? 2 : 1) * N : 0;
}
template <bool GATED>
cudaError_t launch_act_bwd(int act, int64_t M, int64_t N, const float* dY, int64_t lddy, const float* Z, int64_t ldz,
                           float* dZ, int64_t lddz, float* dbias, float* scratch, int sm_count, cudaStream_t s) {
    if (N == 0) return cudaSuccess;
    const int64_t width = (GATED ? 2 : 1) * N;
    if (M == 0) return dbias ? cudaMemsetAsync(dbias, 0, width * sizeof(float), s) : cudaSuccess;
    const RowGrid g = row_grid(M, N, sm_count);
    const bool vec = (N & 3) == 0 && vec4_ok(dY, lddy) && (!Z || (vec4_ok(Z, ldz) && vec4_ok(dZ, lddz)));
    float* partial = dbias ? scratch : nullptr;
    cudaGetLastError();
    if (vec)
        act_bwd_kernel<GATED, true><<<g.grid, dim3(32, kWarps), 0, s>>>(act, M, N, g.rows_per, dY, lddy, Z, ldz, dZ, lddz, partial);
    else
        act_bwd_kernel<GATED, false><<<g.grid, dim3(32, kWarps), 0, s>>>(act, M, N, g.rows_per, dY, lddy, Z, ldz, dZ, lddz, partial);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !dbias) return e;
    return launch_sum_partials(partial, g.chunks, width, width, dbias, nullptr, s);
}

bool valid_act(emu_act_t act) { return act >= EMU_ACT_NONE && act <= EMU_ACT_SILU; }
bool size_ok(int64_t v) { return v <= INT32_MAX - 256; }
emu_status_t launched(cudaError_t e) { return e == cudaSuccess ? EMU_STATUS_SUCCESS : EMU_STATUS_LAUNCH_FAILED; }

#define EMU_TRY(expr)                                        \
    do {                                                     \
        const emu_status_t st_ = (expr);                     \
        if (st_ != EMU_STATUS_SUCCESS) return st_;           \
    } while (0)

// A linear layer's products: Y = X W^T + b, dX = dZ W, dW = dZ^T X.
Gemm forward_product(int64_t M, int64_t N, int64_t K, const float* X, int64_t ldx, const float* W, int64_t ldw,
                     const float* bias, float* Y, int64_t ldy) {
    return {false, false, M, N, K, X, ldx, W, ldw, 0.0f, Y, ldy, bias};
}
Gemm input_product(int64_t M, int64_t N, int64_t K, const float* dZ, int64_t lddz, const float* W, int64_t ldw,
                   float* dX, int64_t lddx) {
    return {false, true, M, K, N, dZ, lddz, W, ldw, 0.0f, dX, lddx, nullptr};
}
Gemm weight_product(int64_t M, int64_t N, int64_t K, const float* dZ, int64_t lddz, const float* X, int64_t ldx,
                    float* dW, int64_t lddw) {
    return {true, true, N, K, M, dZ, lddz, X, ldx, 0.0f, dW, lddw, nullptr};
}

emu_status_t linear_act_fwd(emu_mode_t mode, int act, int64_t M, int64_t N, int64_t K, const float* X, int64_t ldx,
                            const float* W, int64_t ldw, const float* bias, const float* R, int64_t ldr, float* Z,
                            int64_t ldz, float* Y, int64_t ldy, const DeviceCtx& dev, cudaStream_t s, bool check) {
    float* out = Z ? Z : Y;
    const int64_t ldo = Z ? ldz : ldy;
    EMU_TRY(gemm(mode, forward_product(M, N, K, X, ldx, W, ldw, bias, out, ldo), s, check));
    if (check || (act == ACT_NONE && !R && !Z)) return EMU_STATUS_SUCCESS;
    return launched(launch_act_fwd<false>(act, M, N, out, ldo, R, ldr, Y, ldy, dev.sm_count, s));
}

emu_status_t gated_fwd(emu_mode_t mode, int act, int64_t M, int64_t F, int64_t K, const float* X, int64_t ldx,
                       const float* W, int64_t ldw, const float* bias, float* Z, int64_t ldz, float* H, int64_t ldh,
                       const DeviceCtx& dev, cudaStream_t s, bool check) {
    EMU_TRY(gemm(mode, forward_product(M, 2 * F, K, X, ldx, W, ldw, bias, Z, ldz), s, check));
    if (check) return EMU_STATUS_SUCCESS;
    return launched(launch_act_fwd<true>(act, M, F, Z, ldz, nullptr, 0, H, ldh, dev.sm_count, s));
}

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" {

emu_status_t emu_linear_act_fwd(emu_mode_t mode, emu_act_t act, int64_t M, int64_t N, int64_t K, const float* X,
                                int64_t ldx, const float* W, int64_t ldw, const float* bias, const float* residual,
                                int64_t ldr, float* Z, int64_t ldz, float* Y, int64_t ldy, emu_stream_t stream) {
    if (!valid_act(act) || M < 0 || N < 0 || K < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0 || N == 0) return EMU_STATUS_SUCCESS;
    if (!Y || ldy < N || (residual && ldr < N) || (Z && ldz < N)) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev{};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    EMU_TRY(linear_act_fwd(mode, act, M, N, K, X, ldx, W, ldw, bias, residual, ldr, Z, ldz, Y, ldy, dev, s, true));
    EMU_TRY(current_device(&dev));
    return linear_act_fwd(mode, act, M, N, K, X, ldx, W, ldw, bias, residual, ldr, Z, ldz, Y, ldy, dev, s, false);
}

emu_status_t emu_linear_act_bwd(emu_mode_t mode, emu_act_t act, int64_t M, int64_t N, int64_t K, const float* dY,
                                int64_t lddy, const float* X, int64_t ldx, const float* W, int64_t ldw, const float* Z,
                                int64_t ldz, float* dZ, int64_t lddz, float* dX, int64_t lddx, float* dW, int64_t lddw,
                                float* dbias, emu_stream_t stream) {
    if (!valid_act(act) || M < 0 || N < 0 || K < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return EMU_STATUS_NOT_SUPPORTED;
    const bool apply = act != EMU_ACT_NONE;
    if (M > 0 && N > 0) {
        if (!dY || lddy < N) return EMU_STATUS_INVALID_VALUE;
        if (apply && (!Z || !dZ || ldz < N || lddz < N)) return EMU_STATUS_INVALID_VALUE;
    }
    const float* G = apply ? dZ : dY;
    const int64_t ldg = apply ? lddz : lddy;
    const Gemm gx = input_product(M, N, K, G, ldg, W, ldw, dX, lddx), gw = weight_product(M, N, K, G, ldg, X, ldx, dW, lddw);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dX) EMU_TRY(gemm(mode, gx, s, true));
    if (dW) EMU_TRY(gemm(mode, gw, s, true));
    DeviceCtx dev;
    EMU_TRY(current_device(&dev));
    float* scratch = nullptr;
    if (dbias) EMU_TRY(reduce_scratch(dev.id, s, column_sum_floats(false, M, N, dev.sm_count), &scratch));
    if (apply || dbias)
        EMU_TRY(launched(launch_act_bwd<false>(act, M, N, dY, lddy, apply ? Z : nullptr, ldz, dZ, lddz, dbias, scratch,
                                               dev.sm_count, s)));
    if (dX) EMU_TRY(gemm(mode, gx, s, false));
    if (dW) EMU_TRY(gemm(mode, gw, s, false));
    return EMU_STATUS_SUCCESS;
}

emu_status_t emu_gated_fwd(emu_mode_t mode, emu_act_t act, int64_t M, int64_t F, int64_t K, const float* X, int64_t ldx,
                           const float* W, int64_t ldw, const float* bias, float* Z, int64_t ldz, float* H, int64_t ldh,
                           emu_stream_t stream) {
    if (!valid_act(act) || M < 0 || F < 0 || K < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(2 * F) || !size_ok(K)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0 || F == 0) return EMU_STATUS_SUCCESS;
    if (!H || ldh < F || !Z || ldz < 2 * F) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev{};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    EMU_TRY(gated_fwd(mode, act, M, F, K, X, ldx, W, ldw, bias, Z, ldz, H, ldh, dev, s, true));
    EMU_TRY(current_device(&dev));
    return gated_fwd(mode, act, M, F, K, X, ldx, W, ldw, bias, Z, ldz, H, ldh, dev, s, false);
}

emu_status_t emu_gated_bwd(emu_mode_t mode, emu_act_t act, int64_t M, int64_t F, int64_t K, const float* dH,
                           int64_t lddh, const float* X, int64_t ldx, const float* W, int64_t ldw, const float* Z,
                           int64_t ldz, float* dZ, int64_t lddz, float* dX, int64_t lddx, float* dW, int64_t lddw,
                           float* dbias, emu_stream_t stream) {
    if (!valid_act(act) || M < 0 || F < 0 || K < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(2 * F) || !size_ok(K)) return EMU_STATUS_NOT_SUPPORTED;
    if (M > 0 && F > 0 && (!dH || !Z || !dZ || lddh < F || ldz < 2 * F || lddz < 2 * F)) return EMU_STATUS_INVALID_VALUE;
    const Gemm gx = input_product(M, 2 * F, K, dZ, lddz, W, ldw, dX, lddx);
    const Gemm gw = weight_product(M, 2 * F, K, dZ, lddz, X, ldx, dW, lddw);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dX) EMU_TRY(gemm(mode, gx, s, true));
    if (dW) EMU_TRY(gemm(mode, gw, s, true));
    DeviceCtx dev;
    EMU_TRY(current_device(&dev));
    float* scratch = nullptr;
    if (dbias) EMU_TRY(reduce_scratch(dev.id, s, column_sum_floats(true, M, F, dev.sm_count), &scratch));
    EMU_TRY(launched(launch_act_bwd<true>(act, M, F, dH, lddh, Z, ldz, dZ, lddz, dbias, scratch, dev.sm_count, s)));
    if (dX) EMU_TRY(gemm(mode, gx, s, false));
    if (dW) EMU_TRY(gemm(mode, gw, s, false));
    return EMU_STATUS_SUCCESS;
}

emu_status_t emu_gated_ffn_fwd(emu_mode_t mode, emu_act_t act, int64_t M, int64_t K, int64_t F, int64_t N,
                               const float* X, int64_t ldx, const float* W_in, int64_t ldwi, const float* b_in,
                               const float* W_out, int64_t ldwo, const float* b_out, const float* residual, int64_t ldr,
                               float* Z, int64_t ldz, float* H, int64_t ldh, float* Y, int64_t ldy, emu_stream_t stream) {
    if (!valid_act(act) || M < 0 || K < 0 || F < 0 || N < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(K) || !size_ok(2 * F) || !size_ok(N)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0) return EMU_STATUS_SUCCESS;
    if (F > 0 && (!H || ldh < F || !Z || ldz < 2 * F)) return EMU_STATUS_INVALID_VALUE;
    if (N > 0 && (!Y || ldy < N || (residual && ldr < N))) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev{};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (const bool check : {true, false}) {
        if (F > 0) EMU_TRY(gated_fwd(mode, act, M, F, K, X, ldx, W_in, ldwi, b_in, Z, ldz, H, ldh, dev, s, check));
        if (N > 0)
            EMU_TRY(linear_act_fwd(mode, ACT_NONE, M, N, F, H, ldh, W_out, ldwo, b_out, residual, ldr, nullptr, 0, Y, ldy,
                                   dev, s, check));
        if (check) EMU_TRY(current_device(&dev));
    }
    return EMU_STATUS_SUCCESS;
}

emu_status_t emu_gated_ffn_bwd(emu_mode_t mode, emu_act_t act, int64_t M, int64_t K, int64_t F, int64_t N,
                               const float* dY, int64_t lddy, const float* X, int64_t ldx, const float* W_in,
                               int64_t ldwi, const float* W_out, int64_t ldwo, const float* Z, int64_t ldz,
                               const float* H, int64_t ldh, float* dZ, int64_t lddz, float* dX, int64_t lddx,
                               float* dW_in, int64_t lddwi, float* db_in, float* dW_out, int64_t lddwo, float* db_out,
                               emu_stream_t stream) {
    if (!valid_act(act) || M < 0 || K < 0 || F < 0 || N < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(K) || !size_ok(2 * F) || !size_ok(N)) return EMU_STATUS_NOT_SUPPORTED;
    if (M > 0 && N > 0 && (!dY || lddy < N)) return EMU_STATUS_INVALID_VALUE;
    if (M > 0 && F > 0 && (!Z || !H || !dZ || ldz < 2 * F || ldh < F || lddz < 2 * F)) return EMU_STATUS_INVALID_VALUE;
    // dH takes the gate half of dZ's storage until dZ replaces it in place
    const Gemm gh = input_product(M, N, F, dY, lddy, W_out, ldwo, dZ, lddz);
    const Gemm go = weight_product(M, N, F, dY, lddy, H, ldh, dW_out, lddwo);
    const Gemm gx = input_product(M, 2 * F, K, dZ, lddz, W_in, ldwi, dX, lddx);
    const Gemm gw = weight_product(M, 2 * F, K, dZ, lddz, X, ldx, dW_in, lddwi);
    const bool inner = dX || dW_in || db_in;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (inner) EMU_TRY(gemm(mode, gh, s, true));
    if (dW_out) EMU_TRY(gemm(mode, go, s, true));
    if (dX) EMU_TRY(gemm(mode, gx, s, true));
    if (dW_in) EMU_TRY(gemm(mode, gw, s, true));
    DeviceCtx dev;
    EMU_TRY(current_device(&dev));
    const size_t n_out = column_sum_floats(false, M, N, dev.sm_count), n_in = column_sum_floats(true, M, F, dev.sm_count);
    float* scratch = nullptr;
    if (db_in || db_out) EMU_TRY(reduce_scratch(dev.id, s, n_out > n_in ? n_out : n_in, &scratch));
    if (dW_out) EMU_TRY(gemm(mode, go, s, false));
    if (db_out)
        EMU_TRY(launched(launch_act_bwd<false>(ACT_NONE, M, N, dY, lddy, nullptr, 0, nullptr, 0, db_out, scratch,
                                               dev.sm_count, s)));
    if (!inner) return EMU_STATUS_SUCCESS;
    EMU_TRY(gemm(mode, gh, s, false));
    EMU_TRY(launched(launch_act_bwd<true>(act, M, F, dZ, lddz, Z, ldz, dZ, lddz, db_in, scratch, dev.sm_count, s)));
    if (dX) EMU_TRY(gemm(mode, gx, s, false));
    if (dW_in) EMU_TRY(gemm(mode, gw, s, false));
    return EMU_STATUS_SUCCESS;
}

}  // extern "C"
