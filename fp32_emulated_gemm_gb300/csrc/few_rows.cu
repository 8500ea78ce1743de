// few_rows.cu -- a layer's forward pass for a few tokens (serving) or a small
// layer.
//
// For a few rows the product is bound by reading the weight once: 4 N K bytes
// for 2 M N K operations.  The emulated kernels' tiles would be nearly empty,
// and splitting them along k to occupy the GPU costs more than the product.
// So a warp takes NR = 4 rows of W whole or, when there are too few of them
// for the GPU, `wk` warps a share of k each, and X comes from L1; a block takes
// up to eight rows of X, further rows are further blocks, whose weights come
// from L2.  Every output is an FP32 sum of fmaf chains, one per lane, added by
// shuffles and then over the shares in order: within the emulated modes'
// bound, and the same bits on every run.
//
// Measured (back to back in a graph, weights in L2; the tiles in brackets):
// one token K = 1024, N = 4096 5.8 us (22.6; 2.5 at the copy rate from memory),
// K = 4096, N = 1024 3.7 us (31.4), gated K = 1024, F = 4096 8.4 us (31.4);
// eight tokens 9.0, 9.0 and 16.0 us; 64 tokens K = 256, N = 1024 8.5 us (14.3),
// K = 1024, N = 4096 56 us (22.8); one token K = 1024, N = 40000, weights from
// memory, 26.7 us (97; 24.2 at the copy rate).  From eight rows on it is bound by L1 and
// the FMAs at 5 TFMA/s; eight weight rows a warp (64 sums a thread) were slower
// (K = 1024, N = 4096, eight tokens: 12.0 us), for they halve the warps.
#include "few_rows.h"

#include "internal.h"
#include "ptx.cuh"
#include "row_ops.cuh"

namespace emu {
namespace {

constexpr int kWarpsPerBlock = 8;

// A float4 of the weight, which no other warp reads: not kept in L1.
__device__ __forceinline__ float4 load_w4(const float* p) {
    float4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}
template <bool VEC> __device__ __forceinline__ float4 load_w(const float* row, int64_t c, int64_t n) {
    if constexpr (VEC) return c < n ? load_w4(row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    else return load4<false, 32>(row, c, n);
}

// Sums of V values over the warp.  Each step hands half of the values to the
// other half of the lanes: V - 1 shuffles and a few instead of 5 V.  Value i ends
// up in v[0] of lanes 32 / V i onwards.
template <int V> __device__ __forceinline__ void warp_sums(float (&v)[V], int lane) {
    static_assert(V <= 32, "at most a value a lane");
    int n = V / 2;
#pragma unroll
    for (int o = 16; o >= 1; o /= 2, n /= 2) {
        const bool hi = lane & o;
        if (n >= 1) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                if (i >= n) break;
                const float keep = hi ? v[i + n] : v[i], give = hi ? v[i] : v[i + n];
                v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
            }
        } else {
            v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
        }
    }
}

// MR: rows of X (M of them real), NR: rows of W per warp (gated: NR / 2 of the
// gate and the same of the up projection), WK: warps that share a row.
template <int MR, int NR, bool GATED, bool VEC, int FAMILY>
__global__ void __launch_bounds__(32 * kWarpsPerBlock) few_rows_kernel(const FewRows p, int wk) {
    constexpr int V = MR * NR, OUT = GATED ? NR / 2 : NR;  // sums of a warp; output columns
    constexpr int U = MR <= 2 ? 4 : 2;                     // steps whose weights are in flight together
    __shared__ float part[kWarpsPerBlock][V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = kWarpsPerBlock / wk, share = warp % wk;
    const int64_t n0 = ((int64_t)blockIdx.x * groups + warp / wk) * OUT;  // first output column
    const int m0 = blockIdx.y * MR, rows = min(MR, p.M - m0);             // this block's rows of X
    if (threadIdx.x == 0) griddep_launch_dependents();
    // this warp's part of k: whole steps of 128
    const int64_t steps = (p.K + 127) / 128, s0 = steps * share / wk, s1 = steps * (share + 1) / wk;
    const int64_t kend = min(p.K, s1 * 128);
    const float* wrow[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        // (columns past the end read the last one's weights and are dropped)
        const int64_t n = min(n0 + j % OUT, p.N - 1) + (GATED && j >= OUT ? p.N : 0);
        wrow[j] = p.W + n * p.ldw;
    }
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    int64_t c = s0 * 128 + (VEC ? 4 * lane : lane);
    float4 w[U][NR];
    auto load = [&](int64_t at) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NR; ++j) w[u][j] = load_w<VEC>(wrow[j], at + 128 * u, kend);
    };
    load(c);
    griddep_wait();  // X may be the previous kernel's
    for (int64_t s = s0; s < s1; s += U, c += 128 * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                if (m >= rows) break;
                const float4 x = load4<VEC, 32>(p.X + (m0 + m) * p.ldx, c + 128 * u, kend);
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    float& a = acc[m * NR + j];
                    a = fmaf(x.x, w[u][j].x, a);
                    a = fmaf(x.y, w[u][j].y, a);
                    a = fmaf(x.z, w[u][j].z, a);
                    a = fmaf(x.w, w[u][j].w, a);
                }
            }
        }
        if (s + U < s1) load(c + 128 * U);
    }
    warp_sums<V>(acc, lane);
    if (lane % (32 / V) == 0) part[warp][lane / (32 / V)] = acc[0];
    __syncthreads();
    // one thread per output: the shares in order, then the epilogue
    for (int t = threadIdx.x; t < groups * MR * OUT; t += 32 * kWarpsPerBlock) {
        const int g = t / (MR * OUT), r = t / OUT % MR, m = m0 + r, j = t % OUT;
        const int64_t n = ((int64_t)blockIdx.x * groups + g) * OUT + j;
        if (r >= rows || n >= p.N) continue;
        auto total = [&](int i) {
            float s = part[g * wk][i];
            for (int k = 1; k < wk; ++k) s += part[g * wk + k][i];
            return s;
        };
        float z = total(r * NR + j), a, d;
        if (p.bias) z += p.bias[n];
        act_value_grad<FAMILY>(p.act, z, a, d);
        float y = a;
        if constexpr (GATED) {
            float u = total(r * NR + OUT + j);
            if (p.bias) u += p.bias[p.N + n];
            y = a * u;
            if (p.D) {
                p.D[m * p.ldd + n] = u * d;
                p.D[m * p.ldd + p.N + n] = a;
            }
        } else {
            if (p.D) p.D[m * p.ldd + n] = d;
            if (p.R) y += p.R[m * p.ldr + n];
        }
        p.Y[m * p.ldy + n] = y;
    }
}

template <int MR, int NR>
cudaError_t launch(const FewRows& p, bool gated, bool after_own, int sm_count, cudaStream_t stream) {
    // 16 warps an SM keep enough of the weight in flight; a share of k is at
    // least one step
    const int out = gated ? NR / 2 : NR;
    const int64_t warps = (p.N + out - 1) / out, steps = (p.K + 127) / 128;
    int wk = 1;
    const int64_t row_groups = (p.M + MR - 1) / MR;
    while (wk < kWarpsPerBlock && row_groups * warps * wk < 16ll * sm_count && 2 * wk <= steps) wk *= 2;
    const int64_t groups = kWarpsPerBlock / wk, grid = (warps + groups - 1) / groups;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    const bool vec = (p.K & 3) == 0 && vec4_ok(p.X, p.M > 1 ? p.ldx : 0) && vec4_ok(p.W, p.ldw);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)row_groups, 1);
    cfg.blockDim = dim3(32 * kWarpsPerBlock, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (after_own && pdl_enabled()) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    cudaError_t e = cudaSuccess;
    for_family(p.act.family, [&](auto fam) {
        constexpr int f = decltype(fam)::value;
        e = gated ? (vec ? cudaLaunchKernelEx(&cfg, few_rows_kernel<MR, NR, true, true, f>, p, wk)
                         : cudaLaunchKernelEx(&cfg, few_rows_kernel<MR, NR, true, false, f>, p, wk))
                  : (vec ? cudaLaunchKernelEx(&cfg, few_rows_kernel<MR, NR, false, true, f>, p, wk)
                         : cudaLaunchKernelEx(&cfg, few_rows_kernel<MR, NR, false, false, f>, p, wk));
    });
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace

bool few_rows_fit(int64_t M, int64_t N, int64_t K) {
    return M <= kFewRowsMax && (double)(M - 8) * (double)N * (double)K <= kFewRowsFma;
}

cudaError_t launch_few_rows(const FewRows& p, bool gated, bool after_own, int sm_count, cudaStream_t stream) {
    if (p.M <= 1) return launch<1, 4>(p, gated, after_own, sm_count, stream);
    if (p.M <= 2) return launch<2, 4>(p, gated, after_own, sm_count, stream);
    if (p.M <= 4) return launch<4, 4>(p, gated, after_own, sm_count, stream);
    return launch<8, 4>(p, gated, after_own, sm_count, stream);  // eight rows a block
}

}  // namespace emu
