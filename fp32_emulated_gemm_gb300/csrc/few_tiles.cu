// few_tiles.cu -- the forward products of some rows in groups on the CUDA cores: for
// more rows a group than few_rows.cu reads from L1 for each, and fewer than fill the
// emulated kernel's 256-row tiles.
//
// A block has MR rows of a group and 128 of its weight's rows (gated: 64 of either
// half); both come through shared memory, 32 values of k at a time, three stages of
// them in flight (a row's stage is padded to 36 words, so that eight rows' 16 bytes
// lie in different banks).  A thread sums MR / 4 x 4 outputs, the even and the odd k
// apart, by two-word FMAs.  Where there are too few blocks for the GPU, those of a
// cluster share the contraction and add their sums, in order, out of one another's
// shared memory.
//
// Gated blocks of 8 experts, K = 1024, F = 4096: 64 rows 128 us (few_rows.cu 148, the
// tiles 252), 128 rows 141 (196, 253), 256 rows 248 (358, 256); 64 experts, K = 512, F =
// 1024: 512 rows 117 (125, 232), 1024 rows 149 (215, 257); 16 experts, K = F = 1024, 256
// rows 85 (110, 150).  Bound by latency at 12 warps an SM: the FMA pipe is busy half of
// the time, shared memory's likewise (32 rows a group, 8 experts).  Neither more and
// shorter shares of a contraction nor 32 rows a block for groups of 8 to 16 gained
// anything; leaving out a partial block's empty rows did (32 rows 129 -> 120 us, 256
// rows 261 -> 248).
#include "few_tiles.h"

#include <type_traits>

#include "group_rows.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "row_ops.cuh"

namespace emu {
namespace {

constexpr int kThreads = 128, kColumns = 128, kStep = 32, kPad = kStep + 4, kStages = 3;
constexpr int kSumPad = kColumns + 8;  // a row of sums: four rows' eight words in different banks

template <int MR> constexpr int kStageFloats = (kColumns + MR) * kPad;
template <int MR> constexpr size_t kSmem = (size_t)kStages * kStageFloats<MR> * sizeof(float);

// `bytes` of 16 from global to shared memory, the rest zeros.
__device__ __forceinline__ void copy16(float* to, const float* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(__cvta_generic_to_global(from)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fma2(uint64_t& c, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
__device__ __forceinline__ float load_cluster(uint32_t local, uint32_t rank) {
    uint32_t remote;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

template <int MR, bool GATED, int FAMILY>
__global__ void __launch_bounds__(kThreads, 3) few_tiles_kernel(const __grid_constant__ FewRows p) {
    extern __shared__ __align__(16) float sh[];
    constexpr int TM = MR / 4, OUT = GATED ? kColumns / 2 : kColumns;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rg = lane >> 3, cg = warp * 8 + (lane & 7);
    if (threadIdx.x == 0) griddep_launch_dependents();
    // (the offsets are there before the kernel that this one may overlap)
    const int3 g = rows_of_block(p.offsets, p.groups, p.M, MR, blockIdx.y);
    const int rows = g.y;
    if (rows <= 0) {  // (all of a cluster)
        griddep_wait();  // the launch ends after the one before it, if no block has rows too
        return;
    }
    const float *X = p.X + g.x * p.ldx, *W = p.W + g.z * ((GATED ? 2 : 1) * p.N * p.ldw);
    const int64_t n0 = blockIdx.x * (int64_t)OUT;
    const int steps = (int)((p.K + kStep - 1) / kStep), shares = gridDim.z, share = blockIdx.z;
    const int s0 = (int)((int64_t)steps * share / shares), s1 = (int)((int64_t)steps * (share + 1) / shares);
    // a thread copies 16 bytes of every 16th row (columns past the end are the last
    // one's and dropped, rows past the end the last one's and not stored)
    const int piece = 4 * (threadIdx.x & 7), first = threadIdx.x >> 3;
    const int N = (int)p.N, K = (int)p.K, c0 = (int)n0 + first;
    const unsigned ldw = (unsigned)p.ldw, ldx = (unsigned)p.ldx;
    auto load_w = [&](int s) {
        float* to = sh + s % kStages * kStageFloats<MR> + first * kPad + piece;
        const int k = s * kStep + piece, bytes = k < K ? 16 : 0;
        const float* from = W + (k < K ? k : 0);
        if (s < s1) {
#pragma unroll
            for (int i = 0; i < kColumns / 16; ++i) {
                const unsigned n = min(c0 + 16 * i % OUT, N - 1) + (GATED && 16 * i >= OUT ? N : 0);
                copy16(to + 16 * i * kPad, from + (uint64_t)n * ldw, bytes);
            }
        }
    };
    auto load_x = [&](int s) {
        float* to = sh + s % kStages * kStageFloats<MR> + (kColumns + first) * kPad + piece;
        const int k = s * kStep + piece, bytes = k < K ? 16 : 0;
        const float* from = X + (k < K ? k : 0);
        if (s < s1) {
#pragma unroll
            for (int i = 0; i < MR / 16; ++i)
                copy16(to + 16 * i * kPad, from + (uint64_t)(unsigned)min(first + 16 * i, rows - 1) * ldx, bytes);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load_w(s0 + i);
    griddep_wait();  // X
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load_x(s0 + i);
    uint64_t acc[TM][4];
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j] = 0;
    // (a block of fewer rows leaves out what would be nobody's)
    auto work = [&](auto M) {
        constexpr int mine = decltype(M)::value;
        for (int s = s0; s < s1; ++s) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncthreads();  // the stage is there, and the last one has been read
            load_w(s + kStages - 1);
            load_x(s + kStages - 1);
            const float* ws = sh + s % kStages * kStageFloats<MR> + cg * kPad;
            const float* xs = sh + s % kStages * kStageFloats<MR> + (kColumns + rg) * kPad;
#pragma unroll
            for (int k = 0; k < kStep; k += 4) {
                ulonglong2 w[4], x[mine];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const ulonglong2*>(ws + 32 * j * kPad + k);
#pragma unroll
                for (int m = 0; m < mine; ++m) x[m] = *reinterpret_cast<const ulonglong2*>(xs + 4 * m * kPad + k);
#pragma unroll
                for (int m = 0; m < mine; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        fma2(acc[m][j], x[m].x, w[j].x);
                        fma2(acc[m][j], x[m].y, w[j].y);
                    }
            }
        }
    };
    if (rows > MR / 2) work(std::integral_constant<int, TM>{});
    else if (rows > MR / 4) work(std::integral_constant<int, TM / 2>{});
    else work(std::integral_constant<int, TM / 4>{});
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // the sums, where the stages were
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sh[(rg + 4 * m) * kSumPad + cg + 32 * j] = __uint_as_float((uint32_t)acc[m][j]) + __uint_as_float((uint32_t)(acc[m][j] >> 32));
    if (shares > 1) cluster_sync(); else __syncthreads();
    auto total = [&](int at) {
        if (shares == 1) return sh[at];
        const uint32_t local = smem_u32(sh + at);
        float v = load_cluster(local, 0);
        for (int q = 1; q < shares; ++q) v += load_cluster(local, q);
        return v;
    };
    for (int i = share * kThreads + threadIdx.x; i < rows * OUT; i += shares * kThreads) {
        const int r = i / OUT, c = i % OUT;
        const int64_t m = g.x + r, n = n0 + c;
        if (n >= p.N) continue;
        float a, d;
        act_value_grad<FAMILY>(p.act, total(r * kSumPad + c), a, d);
        if constexpr (GATED) {
            const float u = total(r * kSumPad + OUT + c);
            if (p.D) {
                p.D[m * p.ldd + n] = u * d;
                p.D[m * p.ldd + p.N + n] = a;
            }
            a *= u;
        }
        p.Y[m * p.ldy + n] = a;
    }
    if (shares > 1) cluster_sync();  // (the others' sums are read until here)
}

template <int MR> cudaError_t launch(const FewRows& p, bool gated, bool after_own, int sm_count, cudaStream_t stream) {
    const int out = gated ? kColumns / 2 : kColumns;
    const int64_t columns = (p.N + out - 1) / out, row_blocks = p.M / MR + (p.M < p.groups ? p.M : p.groups);
    if (columns > INT32_MAX || row_blocks > 65535) return cudaErrorInvalidConfiguration;
    // blocks for every place of the three that an SM holds, if each has 128 values of k
    const int64_t busy = columns * (p.M / MR > p.groups ? p.M / MR : p.M < p.groups ? p.M : p.groups);
    int shares = 1;
    while (shares < 8 && 2 * busy * shares <= 3 * (int64_t)sm_count && p.K >= 256 * shares) shares *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)columns, (unsigned)row_blocks, (unsigned)shares);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem<MR>;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = (unsigned)shares;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_own && pdl_enabled() ? 2 : 1;
    cudaError_t e = cudaErrorInvalidValue;
    auto run = [&](auto kernel) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem<MR>);
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, p);
    };
    for_family(p.act.family, [&](auto fam) {
        constexpr int f = decltype(fam)::value;
        if (gated) run(few_tiles_kernel<MR, true, f>);
        else if constexpr (f == FAMILY_LINEAR) run(few_tiles_kernel<MR, false, f>);  // (the output projection: no activation)
    });
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace

bool few_tiles_fit(const FewRows& p) {
    return (p.K & 3) == 0 && p.ldx <= INT32_MAX && p.ldw <= INT32_MAX && vec4_ok(p.X, p.M > 1 ? p.ldx : 0) && vec4_ok(p.W, p.ldw);
}

cudaError_t launch_few_tiles(const FewRows& p, bool gated, bool after_own, int sm_count, cudaStream_t stream) {
    if (!few_tiles_fit(p)) return cudaErrorMisalignedAddress;
    // (a block's rows: about what a group has)
    return p.M <= 16 * (int64_t)p.groups ? launch<16>(p, gated, after_own, sm_count, stream)
                                         : launch<32>(p, gated, after_own, sm_count, stream);
}

}  // namespace emu
