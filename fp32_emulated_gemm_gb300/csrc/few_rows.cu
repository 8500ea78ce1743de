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

#include <type_traits>

#include "group_rows.cuh"
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
template <int MR, int NR, bool GATED, bool VEC, int FAMILY, bool GROUPED = false>
__global__ void __launch_bounds__(32 * kWarpsPerBlock) few_rows_kernel(const FewRows p, int wk) {
    constexpr int V = MR * NR, OUT = GATED ? NR / 2 : NR;  // sums of a warp; output columns
    constexpr int U = MR <= 2 ? 4 : 2;                     // steps whose weights are in flight together
    __shared__ float part[kWarpsPerBlock][V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = kWarpsPerBlock / wk, share = warp % wk;
    const int64_t n0 = ((int64_t)blockIdx.x * groups + warp / wk) * OUT;  // first output column
    int m0 = blockIdx.y * MR, rows = min(MR, p.M - m0);                   // this block's rows of X
    const float* W = p.W;
    if (threadIdx.x == 0) griddep_launch_dependents();
    if constexpr (GROUPED) {
        // (the offsets are there before the kernel that this one may overlap)
        const int3 g = rows_of_block(p.offsets, p.groups, p.M, MR, blockIdx.y);
        if (g.y <= 0) {
            griddep_wait();  // the launch ends after the one before it, if no block has rows too
            return;
        }
        m0 = g.x;
        rows = g.y;
        W += g.z * ((GATED ? 2 : 1) * p.N * p.ldw);
    }
    // this warp's part of k: whole steps of 128
    const int64_t steps = (p.K + 127) / 128, s0 = steps * share / wk, s1 = steps * (share + 1) / wk;
    const int64_t kend = min(p.K, s1 * 128);
    const float* wrow[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        // (columns past the end read the last one's weights and are dropped)
        const int64_t n = min(n0 + j % OUT, p.N - 1) + (GATED && j >= OUT ? p.N : 0);
        wrow[j] = W + n * p.ldw;
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

// Rows in groups with work for every warp of the GPU: a warp takes whole rows of
// its group's weight, four at a time, one lot after the other, and asks for the next
// steps' weights across the lots, so that loads are always in flight; a block's rows
// of X come from L1.  The same sums in the same order as above with wk = 1.
// Gated blocks of 8 experts, K = 1024, F = 4096 (both products; 59 us at the copy rate
// for their weights): 16 rows 68 us, 64 rows 128, 128 rows 215, where a lot a warp
// above takes 94, 205 and 366 us; 64 experts, K = 512, F = 1024 (59 us), 512 rows 129
// and 241.  With few lots the form above keeps more warps busy: 2 rows 34 and 22 us, 4
// rows 44 and 39.
template <int MR, bool GATED, bool VEC, int FAMILY>
__global__ void __launch_bounds__(32 * kWarpsPerBlock, 2) few_rows_stream_kernel(const FewRows p, int lots) {
    constexpr int NR = 4, V = MR * NR, OUT = GATED ? NR / 2 : NR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) griddep_launch_dependents();
    // (the offsets are there before the kernel that this one may overlap)
    const int3 g = rows_of_block(p.offsets, p.groups, p.M, MR, blockIdx.y);
    const int rows = g.y;
    if (rows <= 0) {
        griddep_wait();  // (as above)
        return;
    }
    const float* X = p.X + g.x * p.ldx + (VEC ? 4 * lane : lane);
    const float* W = p.W + g.z * ((GATED ? 2 : 1) * p.N * p.ldw) + (VEC ? 4 * lane : lane);
    const int64_t last = (p.N + OUT - 1) / OUT;                                        // lots of the weight
    const int64_t l0 = (int64_t)blockIdx.x * lots + warp, l1 = min((int64_t)(blockIdx.x + 1) * lots, last);
    const int steps = (int)((p.K + 127) / 128);
    float4 w[2][NR];
    // the weights of step s of lot l, and the step after it
    int64_t ahead_lot = l0;
    int ahead_step = 0;
    const float* row[NR];
    auto rows_of_lot = [&] {
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            // (columns past the end read the last one's weights and are dropped)
            const int64_t n = min(ahead_lot * OUT + j % OUT, p.N - 1) + (GATED && j >= OUT ? p.N : 0);
            row[j] = W + n * p.ldw;
        }
    };
    rows_of_lot();
    const int64_t kl = p.K - (VEC ? 4 * lane : lane);  // this lane's columns end there
    auto load = [&](float4 (&v)[NR]) {
        if (ahead_lot >= l1) return;
        const int64_t at = 128 * (int64_t)ahead_step;
#pragma unroll
        for (int j = 0; j < NR; ++j) v[j] = load_w<VEC>(row[j], at, kl);
        if (++ahead_step == steps) {
            ahead_step = 0;
            ahead_lot += kWarpsPerBlock;
            rows_of_lot();
        }
    };
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    int64_t lot = l0;
    int step = 0;
    auto work = [&](float4 (&v)[NR]) {
        const int64_t at = 128 * (int64_t)step;
        constexpr int B = MR < 4 ? MR : 4;  // rows of X loaded together
#pragma unroll
        for (int m0 = 0; m0 < MR; m0 += B) {
            if (m0 >= rows) break;
            float4 x[B];
#pragma unroll
            for (int m = 0; m < B; ++m) x[m] = load4<VEC, 32>(X + (m0 + m) * p.ldx, at, m0 + m < rows ? kl : 0);
#pragma unroll
            for (int m = 0; m < B; ++m)
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    float& a = acc[(m0 + m) * NR + j];
                    a = fmaf(x[m].x, v[j].x, a);
                    a = fmaf(x[m].y, v[j].y, a);
                    a = fmaf(x[m].z, v[j].z, a);
                    a = fmaf(x[m].w, v[j].w, a);
                }
        }
        load(v);
        if (++step < steps) return;
        // the lot's outputs: value i in the lanes from 32 / V i on
        warp_sums<V>(acc, lane);
        const int i = lane / (32 / V), r = i / NR, j = i % NR;
        const int64_t n = lot * OUT + j;
        float z = acc[0], a, d;
        act_value_grad<FAMILY>(p.act, z, a, d);
        const float u = GATED ? __shfl_down_sync(0xFFFFFFFFu, z, OUT * (32 / V)) : 0.f;
        if (lane % (32 / V) == 0 && r < rows && j < OUT && n < p.N) {
            const int64_t m = g.x + r;
            if constexpr (GATED) {
                if (p.D) {
                    p.D[m * p.ldd + n] = u * d;
                    p.D[m * p.ldd + p.N + n] = a;
                }
                p.Y[m * p.ldy + n] = a * u;
            } else {
                p.Y[m * p.ldy + n] = a;
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
        step = 0;
        lot += kWarpsPerBlock;
    };
    load(w[0]);
    load(w[1]);
    griddep_wait();  // X may be the previous kernel's
    while (lot < l1) {
        work(w[0]);
        if (lot < l1) work(w[1]);
    }
}

template <int MR>
cudaError_t launch_stream(const FewRows& p, bool gated, bool after_own, int sm_count, cudaStream_t stream) {
    const int out = gated ? 2 : 4;
    const int64_t row_blocks = p.M / MR + (p.M < p.groups ? p.M : p.groups), all = (p.N + out - 1) / out;
    // about three turns of the two blocks that an SM holds
    int64_t lots = all * row_blocks / ((int64_t)sm_count * 6);
    lots = lots < kWarpsPerBlock ? kWarpsPerBlock : (lots + kWarpsPerBlock - 1) / kWarpsPerBlock * kWarpsPerBlock;
    const int64_t grid = (all + lots - 1) / lots;
    if (grid > INT32_MAX || row_blocks > 65535) return cudaErrorInvalidConfiguration;
    const bool vec = (p.K & 3) == 0 && vec4_ok(p.X, p.M > 1 ? p.ldx : 0) && vec4_ok(p.W, p.ldw);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)row_blocks, 1);
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
        if (gated) e = vec ? cudaLaunchKernelEx(&cfg, few_rows_stream_kernel<MR, true, true, f>, p, (int)lots)
                           : cudaLaunchKernelEx(&cfg, few_rows_stream_kernel<MR, true, false, f>, p, (int)lots);
        else if constexpr (f == FAMILY_LINEAR)  // (the output projection: no activation)
            e = vec ? cudaLaunchKernelEx(&cfg, few_rows_stream_kernel<MR, false, true, f>, p, (int)lots)
                    : cudaLaunchKernelEx(&cfg, few_rows_stream_kernel<MR, false, false, f>, p, (int)lots);
        else e = cudaErrorInvalidValue;
    });
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

template <int MR, int NR, bool GROUPED = false>
cudaError_t launch(const FewRows& p, bool gated, bool after_own, int sm_count, cudaStream_t stream) {
    // 16 warps an SM keep enough of the weight in flight; a share of k is at
    // least one step
    const int out = gated ? NR / 2 : NR;
    const int64_t warps = (p.N + out - 1) / out, steps = (p.K + 127) / 128;
    int wk = 1;
    // (every group's last block may be partial)
    const int64_t row_groups = GROUPED ? p.M / MR + (p.M < p.groups ? p.M : p.groups) : (p.M + MR - 1) / MR;
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
        e = gated ? (vec ? cudaLaunchKernelEx(&cfg, few_rows_kernel<MR, NR, true, true, f, GROUPED>, p, wk)
                         : cudaLaunchKernelEx(&cfg, few_rows_kernel<MR, NR, true, false, f, GROUPED>, p, wk))
                  : (vec ? cudaLaunchKernelEx(&cfg, few_rows_kernel<MR, NR, false, true, f, GROUPED>, p, wk)
                         : cudaLaunchKernelEx(&cfg, few_rows_kernel<MR, NR, false, false, f, GROUPED>, p, wk));
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

cudaError_t launch_few_rows_grouped(const FewRows& p, bool gated, bool streaming, bool after_own, int sm_count,
                                    cudaStream_t stream) {
    auto form = [&](auto MR) {
        constexpr int mr = decltype(MR)::value;
        return streaming ? launch_stream<mr>(p, gated, after_own, sm_count, stream)
                         : launch<mr, 4, true>(p, gated, after_own, sm_count, stream);
    };
    // (a block's rows: about what a group has)
    const int64_t m = p.M, g = p.groups;
    if (4 * m <= g) return form(std::integral_constant<int, 1>{});
    if (m <= g) return form(std::integral_constant<int, 2>{});
    if (m <= 3 * g) return form(std::integral_constant<int, 4>{});
    return form(std::integral_constant<int, 8>{});
}

}  // namespace emu
