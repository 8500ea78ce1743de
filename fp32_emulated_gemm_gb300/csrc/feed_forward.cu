// feed_forward.cu -- the feed-forward operators around the emulated products:
// a linear layer with bias, activation and residual, and the gated
// feed-forward block, each with its backward pass.
//
//   linear_act: Z = X W^T + b, Y = a(Z) + R;              D = a'(Z)
//               dZ = dY D, dX = dZ W, dW = dZ^T X, db = sum over rows of dZ
//   gated:      [G | U] = X [Wg; Wu]^T + [bg | bu], H = a(G) U;  D = [U a'(G) | a(G)]
//               dZ = [dH | dH] D, then as above
//   gated_ffn:  Y = H Wo^T + bo + R;  dH = dY Wo, dWo = dY^T H, dbo = sum of dY
// The forward pass stores the factors D for the backward pass when asked to.
#include <cuda_runtime.h>

#include "activation.cuh"
#include "aligned.cuh"
#include "few_rows.h"
#include "internal.h"
#include "row_ops.cuh"

namespace emu {
namespace {

// The row-wise kernels: a warp covers 128 columns (a float4 per lane, or four
// words 32 apart where rows are not 16-byte aligned) of one row at a time, the
// eight warps of a block take rows in turn, and a block has one chunk of rows.
// They are bound by memory: the gated backward kernel with its sums, 65536 x
// 1024 (1.34 GB), 215 us, 92% of the copy rate.
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

// Y = a(Z) + R and D = a'(Z), or with GATED Y = a(G) U and D = [U a'(G) | a(G)]
// from Z = [G | U] of 2N columns.  D may be null, and Y or D may be Z itself.
template <bool GATED, bool VEC, int FAMILY>
__global__ void __launch_bounds__(32 * kWarps)
act_fwd_kernel(ActParams act, int64_t M, int64_t N, int64_t rows_per, const float* Z, int64_t ldz, const float* R,
               int64_t ldr, float* D, int64_t ldd, float* Y, int64_t ldy) {
    constexpr int S = 32;
    const int64_t c = blockIdx.x * (int64_t)kCols + (VEC ? 4 * threadIdx.x : threadIdx.x);
    const int64_t r1 = min(M, (blockIdx.y + 1) * rows_per);
    for (int64_t r = blockIdx.y * rows_per + threadIdx.y; r < r1; r += kWarps) {
        const float4 z = load4<VEC, S>(Z + r * ldz, c, N);
        float4 a, d;
        act_value_grad4<FAMILY>(act, z, a, d);
        float4 y = a;
        if constexpr (GATED) {
            const float4 u = load4<VEC, S>(Z + r * ldz + N, c, N);
            y = make_float4(a.x * u.x, a.y * u.y, a.z * u.z, a.w * u.w);
            d = make_float4(d.x * u.x, d.y * u.y, d.z * u.z, d.w * u.w);
            if (D) store4<VEC, S>(D + r * ldd + N, c, N, a);
        } else if (R) {
            const float4 q = load4<VEC, S>(R + r * ldr, c, N);
            y = make_float4(y.x + q.x, y.y + q.y, y.z + q.z, y.w + q.w);
        }
        if (D) store4<VEC, S>(D + r * ldd, c, N, d);
        store4<VEC, S>(Y + r * ldy, c, N, y);
    }
}

// Four columns' sums of the block's eight warps, added in order, to out[c ..].
template <bool VEC>
__device__ __forceinline__ void store_block_sums(float4 (&sums)[kWarps][32], float* out, int64_t c, int64_t n) {
    float4 t = sums[0][threadIdx.x];
    for (int i = 1; i < kWarps; ++i) {
        const float4 v = sums[i][threadIdx.x];
        t = make_float4(t.x + v.x, t.y + v.y, t.z + v.z, t.w + v.w);
    }
    // (partial rows of odd width: word stores)
    constexpr int W = VEC ? 1 : 32;
    if (c < n) out[c] = t.x;
    if (c + W < n) out[c + W] = t.y;
    if (c + 2 * W < n) out[c + 2 * W] = t.z;
    if (c + 3 * W < n) out[c + 3 * W] = t.w;
}

// dZ = dY D, or with GATED dZ = [dY | dY] D (2N columns); the sums of this
// block's rows of dZ go to partial[blockIdx.y].  dZ may take dY's place.
template <bool GATED, bool VEC>
__global__ void __launch_bounds__(32 * kWarps)
act_bwd_kernel(int64_t M, int64_t N, int64_t rows_per, const float* dY, int64_t lddy, const float* D, int64_t ldd,
               float* dZ, int64_t lddz, float* partial) {
    constexpr int S = 32;
    __shared__ float4 sums[GATED ? 2 : 1][kWarps][32];
    const int64_t c = blockIdx.x * (int64_t)kCols + (VEC ? 4 * threadIdx.x : threadIdx.x);
    const int64_t r1 = min(M, (blockIdx.y + 1) * rows_per);
    float4 sg = make_float4(0.f, 0.f, 0.f, 0.f), su = sg;
    for (int64_t r = blockIdx.y * rows_per + threadIdx.y; r < r1; r += kWarps) {
        float4 g = load4<VEC, S>(dY + r * lddy, c, N);
        const float4 d = load4<VEC, S>(D + r * ldd, c, N);
        if constexpr (GATED) {
            const float4 a = load4<VEC, S>(D + r * ldd + N, c, N);
            const float4 du = make_float4(g.x * a.x, g.y * a.y, g.z * a.z, g.w * a.w);
            store4<VEC, S>(dZ + r * lddz + N, c, N, du);
            su = make_float4(su.x + du.x, su.y + du.y, su.z + du.z, su.w + du.w);
        }
        g = make_float4(g.x * d.x, g.y * d.y, g.z * d.z, g.w * d.w);
        store4<VEC, S>(dZ + r * lddz, c, N, g);
        sg = make_float4(sg.x + g.x, sg.y + g.y, sg.z + g.z, sg.w + g.w);
    }
    if (!partial) return;
    if (threadIdx.x == 0 && threadIdx.y == 0) griddep_launch_dependents();
    sums[0][threadIdx.y][threadIdx.x] = sg;
    if constexpr (GATED) sums[1][threadIdx.y][threadIdx.x] = su;
    __syncthreads();
    if (threadIdx.y < (GATED ? 2 : 1))
        store_block_sums<VEC>(sums[threadIdx.y], partial + blockIdx.y * ((GATED ? 2 : 1) * N) + threadIdx.y * N, c, N);
}

// Sums of a matrix's columns over chunks of its rows: partial[chunk][column].
struct SumJob {
    const float* A;
    int64_t lda, M, N, rows_per;
    int col_blocks;
    float* partial;
};
template <bool VEC>
__global__ void __launch_bounds__(32 * kWarps) column_sums_kernel(const SumJob a) {
    constexpr int S = 32;
    __shared__ float4 sums[kWarps][32];
    const int64_t chunk = blockIdx.x / a.col_blocks;
    const int64_t c = (blockIdx.x % a.col_blocks) * (int64_t)kCols + (VEC ? 4 * threadIdx.x : threadIdx.x);
    const int64_t r1 = min(a.M, (chunk + 1) * a.rows_per);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int64_t r = chunk * a.rows_per + threadIdx.y; r < r1; r += kWarps) {
        const float4 v = load4<VEC, S>(a.A + r * a.lda, c, a.N);
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
    if (threadIdx.x == 0 && threadIdx.y == 0) griddep_launch_dependents();
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0) store_block_sums<VEC>(sums, a.partial + chunk * a.N, c, a.N);
}

// p ascending in 32 interleaved chains, which are then added in order: the
// sums do not depend on timing.  Block: 32 columns x 32 chains.  A few hundred
// rows of partial sums take 2 to 3 us, mostly the launch, which overlaps the
// end of the kernel before it.
struct PartialsPair { Partials set[2]; unsigned first_blocks; };
__global__ void __launch_bounds__(1024) sum_partials_kernel(const __grid_constant__ PartialsPair pair) {
    __shared__ float part[32][33];
    const bool second = blockIdx.x >= pair.first_blocks;
    const Partials a = second ? pair.set[1] : pair.set[0];
    const int64_t c = (blockIdx.x - (second ? pair.first_blocks : 0)) * 32ll + threadIdx.x;
    griddep_wait();
    float s = 0.f;
    if (c < a.C) {
        for (int p = threadIdx.y; p < a.P; p += 32) s += a.p[(int64_t)p * a.C + c];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < a.C) {
        float t = part[0][threadIdx.x];
        for (int i = 1; i < 32; ++i) t += part[i][threadIdx.x];
        if (c < a.split) { if (a.out0) a.out0[c] = t; }
        else if (a.out1) a.out1[c - a.split] = t;
    }
}

}  // namespace

cudaError_t launch_sum_partials(const Partials* sets, int n, cudaStream_t stream) {
    PartialsPair pair{};
    unsigned blocks = 0;
    for (int i = 0; i < n; ++i) {
        pair.set[i] = sets[i];
        blocks += (unsigned)((sets[i].C + 31) / 32);
        if (i == 0) pair.first_blocks = blocks;
    }
    if (blocks == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, 1, 1);
    cfg.blockDim = dim3(32, 32, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, sum_partials_kernel, pair);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

namespace {

template <bool GATED>
cudaError_t launch_act_fwd(int act, int64_t M, int64_t N, const float* Z, int64_t ldz, const float* R, int64_t ldr,
                           float* D, int64_t ldd, float* Y, int64_t ldy, int sm_count, cudaStream_t s) {
    if (M == 0 || N == 0) return cudaSuccess;
    const RowGrid g = row_grid(M, N, sm_count);
    const bool vec = (N & 3) == 0 && vec4_ok(Z, ldz) && vec4_ok(Y, ldy) && (!R || vec4_ok(R, ldr)) && (!D || vec4_ok(D, ldd));
    cudaGetLastError();
    const ActParams ap = act_params(act);
    for_family(ap.family, [&](auto fam) {
        constexpr int f = decltype(fam)::value;
        const dim3 block(32, kWarps);
        if (vec) act_fwd_kernel<GATED, true, f><<<g.grid, block, 0, s>>>(ap, M, N, g.rows_per, Z, ldz, R, ldr, D, ldd, Y, ldy);
        else act_fwd_kernel<GATED, false, f><<<g.grid, block, 0, s>>>(ap, M, N, g.rows_per, Z, ldz, R, ldr, D, ldd, Y, ldy);
    });
    return cudaGetLastError();
}

// `scratch`: act_bwd_floats() floats when dbias is wanted, else null
size_t act_bwd_floats(bool gated, int64_t M, int64_t N, int sm_count) {
    return M > 0 && N > 0 ? (size_t)row_grid(M, N, sm_count).chunks * (gated ? 2 : 1) * N : 0;
}
template <bool GATED>
cudaError_t launch_act_bwd(int64_t M, int64_t N, const float* dY, int64_t lddy, const float* D, int64_t ldd, float* dZ,
                           int64_t lddz, float* dbias, float* scratch, int sm_count, cudaStream_t s) {
    if (N == 0) return cudaSuccess;
    const int64_t width = (GATED ? 2 : 1) * N;
    if (M == 0) return dbias ? cudaMemsetAsync(dbias, 0, width * sizeof(float), s) : cudaSuccess;
    const RowGrid g = row_grid(M, N, sm_count);
    const bool vec = (N & 3) == 0 && vec4_ok(dY, lddy) && vec4_ok(D, ldd) && vec4_ok(dZ, lddz);
    float* partial = dbias ? scratch : nullptr;
    cudaGetLastError();
    const dim3 block(32, kWarps);
    if (vec) act_bwd_kernel<GATED, true><<<g.grid, block, 0, s>>>(M, N, g.rows_per, dY, lddy, D, ldd, dZ, lddz, partial);
    else act_bwd_kernel<GATED, false><<<g.grid, block, 0, s>>>(M, N, g.rows_per, dY, lddy, D, ldd, dZ, lddz, partial);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !dbias) return e;
    const Partials sums{partial, g.chunks, width, width, dbias, nullptr};
    return launch_sum_partials(&sums, 1, s);
}

// The column sums of a matrix and, in the same two launches, of a second one
// that is narrow in rows already (the partial sums of a product's epilogue:
// dense, at most kDirectRows rows; its out may be null).  scratch:
// column_sums_floats(M, N).
constexpr int64_t kDirectRows = 512;
size_t column_sums_floats(int64_t M, int64_t N, int sm_count) { return act_bwd_floats(false, M, N, sm_count); }
cudaError_t launch_column_sums(const float* A, int64_t lda, int64_t M, int64_t N, float* out, const Partials* direct,
                               float* scratch, int sm_count, cudaStream_t s) {
    Partials sets[2];
    int n = 0;
    if (out && N > 0) {
        if (M == 0) {
            const cudaError_t e = cudaMemsetAsync(out, 0, N * sizeof(float), s);
            if (e != cudaSuccess) return e;
        } else {
            const RowGrid g = row_grid(M, N, sm_count);
            const SumJob job{A, lda, M, N, g.rows_per, (int)g.grid.x, scratch};
            cudaGetLastError();
            const unsigned blocks = g.grid.x * g.grid.y;
            if ((N & 3) == 0 && vec4_ok(A, lda)) column_sums_kernel<true><<<blocks, dim3(32, kWarps), 0, s>>>(job);
            else column_sums_kernel<false><<<blocks, dim3(32, kWarps), 0, s>>>(job);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            sets[n++] = {scratch, g.chunks, N, N, out, nullptr};
        }
    }
    if (direct) sets[n++] = *direct;
    return n ? launch_sum_partials(sets, n, s) : cudaSuccess;
}

bool valid_act(emu_act_t act) { return act >= EMU_ACT_NONE && act <= EMU_ACT_SILU; }
bool size_ok(int64_t v) { return v <= INT32_MAX - 256; }

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

// A few rows go to the CUDA cores in the modes whose bound that meets (FP32 mode
// keeps its one chain per output, the comparators their errors).
bool few_rows(emu_mode_t mode, int64_t M, int64_t N, int64_t K) { return fused_mode(mode) && few_rows_fit(M, N, K); }

// D and the residual of a product's epilogue: 16-byte rows, like C.
bool aligned_rows(const float* p, int64_t ld) { return !p || vec4_ok(p, ld); }

emu_status_t linear_act_fwd(emu_mode_t mode, int act, int64_t M, int64_t N, int64_t K, const float* X, int64_t ldx,
                            const float* W, int64_t ldw, const float* bias, const float* R, int64_t ldr, float* D,
                            int64_t ldd, float* Y, int64_t ldy, const DeviceCtx& dev, cudaStream_t s, Until until,
                            bool after_own = false) {
    if (few_rows(mode, M, N, K)) {
        if (K > 0 && (!X || !W || ldx < K || ldw < K)) return EMU_STATUS_INVALID_VALUE;
        if (until != UNTIL_LAUNCHED) return EMU_STATUS_SUCCESS;
        return launched(launch_few_rows({(int)M, N, K, X, ldx, W, ldw, bias, R, ldr, D, ldd, Y, ldy, act_params(act)}, false,
                                        after_own, dev.sm_count, s));
    }
    if (!aligned_rows(D, ldd) || !aligned_rows(R, ldr)) return EMU_STATUS_NOT_SUPPORTED;
    Gemm g = forward_product(M, N, K, X, ldx, W, ldw, bias, Y, ldy);
    const Fused f{FUSED_ACT, act, R, ldr, D, ldd, nullptr};
    const bool plain = act == ACT_NONE && !R && !D, fuse = fused_mode(mode) && K > 0 && !plain;
    if (fuse) g.fused = &f;
    EMU_TRY(gemm(mode, g, s, until));
    if (until != UNTIL_LAUNCHED || plain || fuse) return EMU_STATUS_SUCCESS;
    return launched(launch_act_fwd<false>(act, M, N, Y, ldy, R, ldr, D, ldd, Y, ldy, dev.sm_count, s));
}

// A mode without a fused epilogue computes [G | U] in D first.
bool gated_needs_d(emu_mode_t mode) { return !fused_mode(mode); }
emu_status_t gated_fwd(emu_mode_t mode, int act, int64_t M, int64_t F, int64_t K, const float* X, int64_t ldx,
                       const float* W, int64_t ldw, const float* bias, float* D, int64_t ldd, float* H, int64_t ldh,
                       const DeviceCtx& dev, cudaStream_t s, Until until) {
    if (few_rows(mode, M, 2 * F, K)) {
        if (K > 0 && (!X || !W || ldx < K || ldw < K)) return EMU_STATUS_INVALID_VALUE;
        if (until != UNTIL_LAUNCHED) return EMU_STATUS_SUCCESS;
        return launched(launch_few_rows({(int)M, F, K, X, ldx, W, ldw, bias, nullptr, 0, D, ldd, H, ldh, act_params(act)},
                                        true, false, dev.sm_count, s));
    }
    if (!aligned_rows(D, ldd)) return EMU_STATUS_NOT_SUPPORTED;
    if (fused_mode(mode) && K > 0) {
        Gemm g = forward_product(M, F, K, X, ldx, W, ldw, bias, H, ldh);
        const Fused f{FUSED_GATED, act, nullptr, 0, D, ldd, nullptr};
        g.fused = &f;
        return gemm(mode, g, s, until);
    }
    if (!D && K == 0) {  // every row is the bias
        if (until != UNTIL_LAUNCHED) return EMU_STATUS_SUCCESS;
        if (bias) return launched(launch_act_fwd<true>(act, M, F, bias, 0, nullptr, 0, nullptr, 0, H, ldh, dev.sm_count, s));
        return launched(cudaMemset2DAsync(H, ldh * sizeof(float), 0, F * sizeof(float), M, s));
    }
    EMU_TRY(gemm(mode, forward_product(M, 2 * F, K, X, ldx, W, ldw, bias, D, ldd), s, until));
    if (until != UNTIL_LAUNCHED) return EMU_STATUS_SUCCESS;
    return launched(launch_act_fwd<true>(act, M, F, D, ldd, nullptr, 0, D, ldd, H, ldh, dev.sm_count, s));
}

// A forward pass in its steps: the arguments' checks, the buffers, then the copies
// of its operands and its launches.
template <class F> emu_status_t in_steps(Aligned& al, DeviceCtx& dev, cudaStream_t s, F pass) {
    al.stand_in();
    EMU_TRY(pass(UNTIL_CHECKED));
    EMU_TRY(current_device(&dev));
    EMU_TRY(al.reserve(s));
    EMU_TRY(pass(UNTIL_RESERVED));
    EMU_TRY(launched(al.launch(s)));
    return pass(UNTIL_LAUNCHED);
}

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" {

int emu_few_rows_query(int64_t M, int64_t N, int64_t K) { return M >= 0 && N >= 0 && K >= 0 && few_rows_fit(M, N, K) ? 1 : 0; }

emu_status_t emu_linear_act_fwd(emu_mode_t mode, emu_act_t act, int64_t M, int64_t N, int64_t K, const float* X,
                                int64_t ldx, const float* W, int64_t ldw, const float* bias, const float* residual,
                                int64_t ldr, float* D, int64_t ldd, float* Y, int64_t ldy, emu_stream_t stream) {
    if (!valid_act(act) || M < 0 || N < 0 || K < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0 || N == 0) return EMU_STATUS_SUCCESS;
    if (!Y || ldy < N || (residual && ldr < N) || (D && ldd < N)) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev{};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    Aligned al;
    if (!few_rows(mode, M, N, K)) {
        al.add(X, ldx, M, K);
        al.add(W, ldw, N, K);
        al.add(residual, ldr, M, N);
        al.add_vector(bias, N);
    }
    return in_steps(al, dev, s, [&](Until until) {
        return linear_act_fwd(mode, act, M, N, K, X, ldx, W, ldw, bias, residual, ldr, D, ldd, Y, ldy, dev, s, until);
    });
}

emu_status_t emu_linear_act_bwd(emu_mode_t mode, int64_t M, int64_t N, int64_t K, const float* dY, int64_t lddy,
                                const float* X, int64_t ldx, const float* W, int64_t ldw, const float* D, int64_t ldd,
                                float* dZ, int64_t lddz, float* dX, int64_t lddx, float* dW, int64_t lddw, float* dbias,
                                emu_stream_t stream) {
    if (M < 0 || N < 0 || K < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return EMU_STATUS_NOT_SUPPORTED;
    const bool rows = M > 0 && N > 0;
    if (rows && (!dY || lddy < N || (D && (!dZ || ldd < N || lddz < N)))) return EMU_STATUS_INVALID_VALUE;
    const bool apply = D && rows;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    Aligned al;  // (D and, with it, dY are not a product's)
    if (!D) al.add(dY, lddy, M, N);
    if (dW) al.add(X, ldx, M, K);
    if (dX) al.add(W, ldw, N, K);
    auto products = [&](Until until) {
        const float* G = D ? dZ : dY;
        const int64_t ldg = D ? lddz : lddy;
        const Gemm gx = input_product(M, N, K, G, ldg, W, ldw, dX, lddx);
        const Gemm gw = weight_product(M, N, K, G, ldg, X, ldx, dW, lddw);
        return gemm_two(mode, dX ? &gx : nullptr, dW ? &gw : nullptr, s, until);
    };
    al.stand_in();
    EMU_TRY(products(UNTIL_CHECKED));
    DeviceCtx dev;
    EMU_TRY(current_device(&dev));
    EMU_TRY(al.reserve(s));
    EMU_TRY(products(UNTIL_RESERVED));
    float* scratch = nullptr;
    if (dbias) EMU_TRY(reduce_scratch(dev.id, s, act_bwd_floats(false, M, N, dev.sm_count), &scratch));
    EMU_TRY(launched(al.launch(s)));
    if (apply)
        EMU_TRY(launched(launch_act_bwd<false>(M, N, dY, lddy, D, ldd, dZ, lddz, dbias, scratch, dev.sm_count, s)));
    else if (dbias)
        EMU_TRY(launched(launch_column_sums(dY, lddy, M, N, dbias, nullptr, scratch, dev.sm_count, s)));
    return products(UNTIL_LAUNCHED);
}

emu_status_t emu_gated_fwd(emu_mode_t mode, emu_act_t act, int64_t M, int64_t F, int64_t K, const float* X, int64_t ldx,
                           const float* W, int64_t ldw, const float* bias, float* D, int64_t ldd, float* H, int64_t ldh,
                           emu_stream_t stream) {
    if (!valid_act(act) || M < 0 || F < 0 || K < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(2 * F) || !size_ok(K)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0 || F == 0) return EMU_STATUS_SUCCESS;
    if (!H || ldh < F || (D && ldd < 2 * F) || (!D && gated_needs_d(mode))) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev{};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    Aligned al;
    if (!few_rows(mode, M, 2 * F, K)) {
        al.add(X, ldx, M, K);
        al.add(W, ldw, 2 * F, K);
        al.add_vector(bias, 2 * F);
    }
    return in_steps(al, dev, s, [&](Until until) {
        return gated_fwd(mode, act, M, F, K, X, ldx, W, ldw, bias, D, ldd, H, ldh, dev, s, until);
    });
}

emu_status_t emu_gated_bwd(emu_mode_t mode, int64_t M, int64_t F, int64_t K, const float* dH, int64_t lddh,
                           const float* X, int64_t ldx, const float* W, int64_t ldw, const float* D, int64_t ldd,
                           float* dZ, int64_t lddz, float* dX, int64_t lddx, float* dW, int64_t lddw, float* dbias,
                           emu_stream_t stream) {
    if (M < 0 || F < 0 || K < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(2 * F) || !size_ok(K)) return EMU_STATUS_NOT_SUPPORTED;
    if (M > 0 && F > 0 && (!dH || !D || !dZ || lddh < F || ldd < 2 * F || lddz < 2 * F)) return EMU_STATUS_INVALID_VALUE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    Aligned al;  // (dH and D are not a product's)
    if (dW) al.add(X, ldx, M, K);
    if (dX) al.add(W, ldw, 2 * F, K);
    auto products = [&](Until until) {
        const Gemm gx = input_product(M, 2 * F, K, dZ, lddz, W, ldw, dX, lddx);
        const Gemm gw = weight_product(M, 2 * F, K, dZ, lddz, X, ldx, dW, lddw);
        return gemm_two(mode, dX ? &gx : nullptr, dW ? &gw : nullptr, s, until);
    };
    al.stand_in();
    EMU_TRY(products(UNTIL_CHECKED));
    DeviceCtx dev;
    EMU_TRY(current_device(&dev));
    EMU_TRY(al.reserve(s));
    EMU_TRY(products(UNTIL_RESERVED));
    float* scratch = nullptr;
    if (dbias) EMU_TRY(reduce_scratch(dev.id, s, act_bwd_floats(true, M, F, dev.sm_count), &scratch));
    EMU_TRY(launched(al.launch(s)));
    EMU_TRY(launched(launch_act_bwd<true>(M, F, dH, lddh, D, ldd, dZ, lddz, dbias, scratch, dev.sm_count, s)));
    return products(UNTIL_LAUNCHED);
}

emu_status_t emu_gated_ffn_fwd(emu_mode_t mode, emu_act_t act, int64_t M, int64_t K, int64_t F, int64_t N,
                               const float* X, int64_t ldx, const float* W_in, int64_t ldwi, const float* b_in,
                               const float* W_out, int64_t ldwo, const float* b_out, const float* residual, int64_t ldr,
                               float* D, int64_t ldd, float* H, int64_t ldh, float* Y, int64_t ldy, emu_stream_t stream) {
    if (!valid_act(act) || M < 0 || K < 0 || F < 0 || N < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(K) || !size_ok(2 * F) || !size_ok(N)) return EMU_STATUS_NOT_SUPPORTED;
    if (M == 0) return EMU_STATUS_SUCCESS;
    if (F > 0 && (!H || ldh < F || (D && ldd < 2 * F) || (!D && gated_needs_d(mode)))) return EMU_STATUS_INVALID_VALUE;
    if (N > 0 && (!Y || ldy < N || (residual && ldr < N))) return EMU_STATUS_INVALID_VALUE;
    DeviceCtx dev{};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    Aligned al;
    if (!few_rows(mode, M, 2 * F, K)) {
        al.add(X, ldx, M, K);
        al.add(W_in, ldwi, 2 * F, K);
        al.add_vector(b_in, 2 * F);
    }
    if (!few_rows(mode, M, N, F)) {
        al.add(W_out, ldwo, N, F);
        al.add(residual, ldr, M, N);
        al.add_vector(b_out, N);
    }
    return in_steps(al, dev, s, [&](Until until) {
        if (F > 0) EMU_TRY(gated_fwd(mode, act, M, F, K, X, ldx, W_in, ldwi, b_in, D, ldd, H, ldh, dev, s, until));
        if (N > 0)
            EMU_TRY(linear_act_fwd(mode, ACT_NONE, M, N, F, H, ldh, W_out, ldwo, b_out, residual, ldr, nullptr, 0, Y, ldy,
                                   dev, s, until, F > 0 && few_rows(mode, M, 2 * F, K)));
        return EMU_STATUS_SUCCESS;
    });
}

emu_status_t emu_gated_ffn_bwd(emu_mode_t mode, int64_t M, int64_t K, int64_t F, int64_t N, const float* dY,
                               int64_t lddy, const float* X, int64_t ldx, const float* W_in, int64_t ldwi,
                               const float* W_out, int64_t ldwo, const float* D, int64_t ldd, const float* H, int64_t ldh,
                               float* dZ, int64_t lddz, float* dX, int64_t lddx, float* dW_in, int64_t lddwi,
                               float* db_in, float* dW_out, int64_t lddwo, float* db_out, emu_stream_t stream) {
    if (M < 0 || K < 0 || F < 0 || N < 0) return EMU_STATUS_INVALID_VALUE;
    if (!size_ok(M) || !size_ok(K) || !size_ok(2 * F) || !size_ok(N)) return EMU_STATUS_NOT_SUPPORTED;
    if (M > 0 && N > 0 && (!dY || lddy < N)) return EMU_STATUS_INVALID_VALUE;
    const bool inner = dX || dW_in || db_in;
    if (M > 0 && F > 0) {
        if (dW_out && (!H || ldh < F)) return EMU_STATUS_INVALID_VALUE;
        if (inner && (!D || !dZ || ldd < 2 * F || lddz < 2 * F)) return EMU_STATUS_INVALID_VALUE;
        if (inner && !aligned_rows(dZ, lddz)) return EMU_STATUS_NOT_SUPPORTED;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    Aligned al;
    if (inner || dW_out) al.add(dY, lddy, M, N);
    if (dW_out) al.add(H, ldh, M, F);
    if (inner) {
        al.add(W_out, ldwo, N, F);
        al.add(D, ldd, M, 2 * F);
    }
    if (dX) al.add(W_in, ldwi, 2 * F, K);
    if (dW_in) al.add(X, ldx, M, K);
    // dZ comes straight from the product's epilogue; or dH takes the gate half
    // of dZ's storage until dZ replaces it in place
    const bool fuse = fused_mode(mode) && N > 0 && M > 0 && F > 0;
    float *scratch = nullptr, *sums = nullptr;
    auto outer_products = [&](Until until) {
        const Fused f{FUSED_GATED_BWD, ACT_NONE, nullptr, 0, const_cast<float*>(D), ldd, fuse && db_in ? sums : nullptr};
        Gemm gh = input_product(M, N, F, dY, lddy, W_out, ldwo, dZ, lddz);
        if (fuse) gh.fused = &f;
        const Gemm go = weight_product(M, N, F, dY, lddy, H, ldh, dW_out, lddwo);
        return gemm_two(mode, inner ? &gh : nullptr, dW_out ? &go : nullptr, s, until);
    };
    auto inner_products = [&](Until until) {
        const Gemm gx = input_product(M, 2 * F, K, dZ, lddz, W_in, ldwi, dX, lddx);
        const Gemm gw = weight_product(M, 2 * F, K, dZ, lddz, X, ldx, dW_in, lddwi);
        return gemm_two(mode, dX ? &gx : nullptr, dW_in ? &gw : nullptr, s, until);
    };
    al.stand_in();
    EMU_TRY(outer_products(UNTIL_CHECKED));
    EMU_TRY(inner_products(UNTIL_CHECKED));
    DeviceCtx dev;
    EMU_TRY(current_device(&dev));
    EMU_TRY(al.reserve(s));
    EMU_TRY(outer_products(UNTIL_RESERVED));
    EMU_TRY(inner_products(UNTIL_RESERVED));
    // Scratch: the output bias's partial sums, the epilogue's (a row for each 32
    // rows) and, where those are many, their own partial sums.
    const int64_t blocks = (M + 31) / 32;
    const bool direct = blocks <= kDirectRows;
    const size_t n_out = column_sums_floats(M, N, dev.sm_count);
    const size_t n_in = !fuse ? act_bwd_floats(true, M, F, dev.sm_count)
                              : (size_t)blocks * 2 * F + (direct ? 0 : column_sums_floats(blocks, 2 * F, dev.sm_count));
    if (db_in || db_out) {
        const size_t out_floats = (n_out + 3) & ~size_t(3);
        EMU_TRY(reduce_scratch(dev.id, s, out_floats + n_in, &scratch));
        sums = scratch + out_floats;
    }
    EMU_TRY(launched(al.launch(s)));
    EMU_TRY(outer_products(UNTIL_LAUNCHED));
    const bool join = fuse && db_in && direct;
    const Partials in_sums{sums, (int)blocks, 2 * F, 2 * F, db_in, nullptr};
    if (db_out || join)
        EMU_TRY(launched(launch_column_sums(dY, lddy, M, N, db_out, join ? &in_sums : nullptr, scratch, dev.sm_count, s)));
    if (!inner) return EMU_STATUS_SUCCESS;
    if (!fuse)
        EMU_TRY(launched(launch_act_bwd<true>(M, F, dZ, lddz, D, ldd, dZ, lddz, db_in, sums, dev.sm_count, s)));
    else if (db_in && !direct)
        EMU_TRY(launched(launch_column_sums(sums, 2 * F, blocks, 2 * F, db_in, nullptr, sums + (size_t)blocks * 2 * F,
                                            dev.sm_count, s)));
    return inner_products(UNTIL_LAUNCHED);
}

}  // extern "C"
