// few_rows_bwd.cu -- the backward products of a few rows in groups, a weight for
// each: dX = dZ W (the weight's rows are the contraction) and dW = dZ^T X.
//
// For a few rows they are bound by reading the weights once and writing their
// gradients, where the emulated kernels' tiles would be nearly empty.
// few_columns: a block has up to eight rows and 128 columns, its warps a share of the
// contraction each; a lane has four columns of all rows, the weight's rows come as
// whole 512-byte lots and the rows' values from L1.  Where that makes too few blocks,
// several share a contraction through a buffer, and a second kernel adds what they
// leave.  The shares are added in order.
// few_sums: a warp has eight rows of C and 128 columns and goes through the group's
// rows in order.  Nobody but the device knows how many those are: an expert that has
// most of them is shared out in chunks, whose sums a second kernel adds in order.  All
// rows on one of 64 experts, K = F = N = 64, 2500 rows: backward pass 1507 us with the
// rows in one chain, 82 in chunks (spread evenly 56 and 58); 256 experts, 12000 rows
// 7190 and 246 (149 and 159); 128 experts, K = F = N = 128, 4096 rows 1776 and 139 (77
// and 82); 64 experts, K = N = 512, F = 1024, 512 rows 454 and 377 (333 and 350).
#include "few_rows_bwd.h"

#include <algorithm>

#include "group_rows.cuh"
#include "internal.h"
#include "row_ops.cuh"

namespace emu {
namespace {

constexpr int kWarps = 8, kColumns = 128, kSumRows = 8;

// Columns c .. c + 3 of a row of n (aligned): the words that exist, else zeros.
// PLAIN: of a matrix that a launch of the same call writes, which this one may
// overlap: the read-only path is for data that nobody writes while the kernel runs,
// also where it is read behind the wait.
template <bool PLAIN = false> __device__ __forceinline__ float4 columns(const float* row, int64_t c, int64_t n) {
    auto load = [](const auto* p) {
        if constexpr (PLAIN) return *p;
        else return __ldg(p);
    };
    if (c + 3 < n) return load(reinterpret_cast<const float4*>(row + c));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < n) v.x = load(row + c);
    if (c + 1 < n) v.y = load(row + c + 1);
    if (c + 2 < n) v.z = load(row + c + 2);
    return v;
}
// (the last columns word by word: what lies behind them is not the output's)
__device__ __forceinline__ void put_columns(float* row, int64_t c, int64_t n, const float4& v) {
    if (c + 3 < n) {
        *reinterpret_cast<float4*>(row + c) = v;
        return;
    }
    if (c < n) row[c] = v.x;
    if (c + 1 < n) row[c + 1] = v.y;
    if (c + 2 < n) row[c + 2] = v.z;
}
__device__ __forceinline__ void fma4(float a, const float4& b, float4& c) {
    c = make_float4(fmaf(a, b.x, c.x), fmaf(a, b.y, c.y), fmaf(a, b.z, c.z), fmaf(a, b.w, c.w));
}

// Columns at .. at + 3 of row r of C.
__device__ __forceinline__ void put_row(const FewColumns& p, int64_t r, int64_t at, const float4& s) {
    float* out = p.C + r * p.ldc;
    if (!p.D) {
        put_columns(out, at, p.N, s);
        return;
    }
    const float* d = p.D + r * p.ldd;
    const float4 f = columns(d, at, p.N);
    put_columns(out, at, p.N, make_float4(s.x * f.x, s.y * f.y, s.z * f.z, s.w * f.w));
    if ((p.N & 3) == 0) {
        const float4 u = columns(d + p.N, at, p.N);
        put_columns(out + p.N, at, p.N, make_float4(s.x * u.x, s.y * u.y, s.z * u.z, s.w * u.w));
    } else {  // (the second half is off the 16-byte boundaries)
        const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + j < p.N) out[p.N + at + j] = v[j] * __ldg(d + p.N + at + j);
    }
}

template <int MR>
__global__ void __launch_bounds__(32 * kWarps, 2) few_columns_kernel(const __grid_constant__ FewColumns p) {
    __shared__ float4 part[kWarps][MR][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) griddep_launch_dependents();
    // (the offsets and the weights are there before the kernel that this one may overlap)
    const int3 g = rows_of_block(p.offsets, p.groups, p.M, MR, blockIdx.y);
    const int rows = g.y;
    const int64_t c = blockIdx.x * (int64_t)kColumns + 4 * lane;
    const float* B = p.B + g.z * (p.K * p.ldb);
    // this warp's share of the contraction, in fours
    const int64_t quads = (p.K + 3) / 4, shares = (int64_t)kWarps * gridDim.z, share = blockIdx.z * kWarps + warp;
    const int64_t q1 = quads * (share + 1) / shares;
    int64_t q = quads * share / shares;
    float4 b[2][4];
    auto load = [&](float4 (&v)[4], int64_t quad) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = rows > 0 && quad < q1 && 4 * quad + j < p.K ? columns(B + (4 * quad + j) * p.ldb, c, p.N)
                                                               : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(b[0], q);
    load(b[1], q + 1);
    griddep_wait();  // A (and what was written before it)
    if (rows <= 0) return;
    const float* A = p.A + g.x * p.lda;
    float4 acc[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) acc[m] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto work = [&](float4 (&v)[4]) {
        constexpr int H = MR < 4 ? MR : 4;  // rows of A loaded together
#pragma unroll
        for (int m0 = 0; m0 < MR; m0 += H) {
            if (m0 >= rows) break;
            float4 a[H];
#pragma unroll
            for (int m = 0; m < H; ++m)
                a[m] = m0 + m < rows ? columns<true>(A + (m0 + m) * p.lda, 4 * q, p.K) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int m = 0; m < H; ++m) {
                fma4(a[m].x, v[0], acc[m0 + m]);
                fma4(a[m].y, v[1], acc[m0 + m]);
                fma4(a[m].z, v[2], acc[m0 + m]);
                fma4(a[m].w, v[3], acc[m0 + m]);
            }
        }
        load(v, q + 2);
        ++q;
    };
    while (q < q1) {
        work(b[0]);
        if (q < q1) work(b[1]);
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) part[warp][m][lane] = acc[m];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * 32; i += 32 * kWarps) {
        const int m = i / 32, l = i % 32;
        float4 s = part[0][m][l];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 v = part[w][m][l];
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        const int64_t r = g.x + m, at = blockIdx.x * (int64_t)kColumns + 4 * l;
        if (gridDim.z > 1) {
            if (at < p.N) *reinterpret_cast<float4*>(p.shares + ((int64_t)blockIdx.z * p.M + r) * p.ldshares + at) = s;
        } else {
            put_row(p, r, at, s);
        }
    }
}

// What the blocks of a contraction left, added.
__global__ void __launch_bounds__(256) add_shares_kernel(const __grid_constant__ FewColumns p, int shares) {
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int begin = min(max(__ldcg(p.offsets), 0), p.M);
    const int end = rows_of_group(p.offsets, p.M, p.groups - 1).y;
    griddep_wait();  // the shares
    const uint32_t quads = (uint32_t)((p.N + 3) / 4);
    const int64_t i = blockIdx.x * 256ll + threadIdx.x, r = i / quads, c = 4 * (i - r * quads);
    if (r < begin || r >= end) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int z = 0; z < shares; ++z) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.shares + ((int64_t)z * p.M + r) * p.ldshares + c));
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
    put_row(p, r, c, s);
}

// PIECES: some group may have more than a chunk of rows.
template <bool PIECES>
__global__ void __launch_bounds__(32 * kWarps) few_sums_kernel(const __grid_constant__ FewSums p, unsigned column_blocks) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) griddep_launch_dependents();
    int2 g;
    if (!PIECES || blockIdx.y < p.groups) {
        g = rows_of_group(p.offsets, p.M, blockIdx.y);
        if constexpr (PIECES) g.y = min(g.y, g.x + p.chunk);
    } else {  // a chunk of the groups' rows behind their first ones
        if (!any_group_above(p.offsets, p.groups, p.M, p.chunk)) {
            griddep_wait();
            return;
        }
        const int3 b = rows_of_block<1>(p.offsets, p.groups, p.M, p.chunk, (int)blockIdx.y - p.groups);
        g = make_int2(b.x, b.x + b.y);
    }
    const int64_t r0 = (int64_t)(blockIdx.x / column_blocks) * (kWarps * kSumRows) + warp * kSumRows;
    const int64_t c = (int64_t)(blockIdx.x % column_blocks) * kColumns + 4 * lane;
    float4 acc[kSumRows];
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    griddep_wait();  // A and B
    if (r0 >= p.R || (PIECES && blockIdx.y >= p.groups && g.y == g.x)) return;
    constexpr int B = 4;  // rows whose loads go out together
    for (int m0 = g.x; m0 < g.y; m0 += B) {
        float4 b[B], a[B], e[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const bool there = m0 + i < g.y;
            const int64_t m = there ? m0 + i : m0;
            b[i] = columns(p.B + m * p.ldb, c, there ? p.N : 0);
            a[i] = columns<true>(p.A + m * p.lda, r0, there ? p.R : 0);
            e[i] = columns<true>(p.A + m * p.lda, r0 + 4, there ? p.R : 0);
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (m0 + i >= g.y) break;
            fma4(a[i].x, b[i], acc[0]);
            fma4(a[i].y, b[i], acc[1]);
            fma4(a[i].z, b[i], acc[2]);
            fma4(a[i].w, b[i], acc[3]);
            fma4(e[i].x, b[i], acc[4]);
            fma4(e[i].y, b[i], acc[5]);
            fma4(e[i].z, b[i], acc[6]);
            fma4(e[i].w, b[i], acc[7]);
        }
    }
    const bool first = !PIECES || blockIdx.y < p.groups;
    float* out = first ? p.C + (blockIdx.y * p.R + r0) * p.ldc : p.pieces + ((blockIdx.y - p.groups) * p.R + r0) * p.ldpieces;
    const int64_t ld = first ? p.ldc : p.ldpieces;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i)
        if (r0 + i < p.R) put_columns(out + i * ld, c, p.N, acc[i]);
}

// The pieces of a group's sums, added to its first chunk's: the blocks of the group's
// first piece do it.  (Both sums of a call in one launch at its end: 2 us less.)
struct TwoSums { FewSums sums[2]; };
__global__ void __launch_bounds__(32 * kWarps) add_pieces_kernel(const __grid_constant__ TwoSums two) {
    const FewSums& p = two.sums[blockIdx.z];
    if (threadIdx.x == 0) griddep_launch_dependents();
    if (!any_group_above(p.offsets, p.groups, p.M, p.chunk)) {
        griddep_wait();
        return;
    }
    const int3 b = rows_of_block<1>(p.offsets, p.groups, p.M, p.chunk, blockIdx.y);
    const int2 g = rows_of_group(p.offsets, p.M, b.z);
    griddep_wait();  // the sums
    if (b.y == 0 || b.x != g.x + p.chunk) return;
    const uint32_t quads = (uint32_t)((p.N + 3) / 4);
    const int n = (g.y - g.x - 1) / p.chunk;
    for (int64_t i = blockIdx.x * (32ll * kWarps) + threadIdx.x; i < p.R * quads; i += gridDim.x * (32ll * kWarps)) {
        const int64_t r = i / quads, c = 4 * (i - r * quads);
        float* out = p.C + (b.z * p.R + r) * p.ldc;
        const float* piece = p.pieces + (blockIdx.y * p.R + r) * p.ldpieces;
        float4 s = columns<true>(out, c, p.N);
#pragma unroll 8
        for (int z = 0; z < n; ++z) {
            const float4 v = columns<true>(piece + z * p.R * p.ldpieces, c, p.N);
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        put_columns(out, c, p.N, s);
    }
}

template <class K, class... Args>
cudaError_t launch(K kernel, dim3 grid, bool after_own, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_own && pdl_enabled() ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace

namespace {
// A block's rows: about what a group has.
int block_rows(int64_t m, int64_t g) { return 4 * m <= g ? 1 : m <= g ? 2 : m <= 3 * g ? 4 : 8; }
int64_t row_blocks(int64_t m, int64_t g) { return m / block_rows(m, g) + (m < g ? m : g); }  // (every group's last may be partial)
int64_t column_blocks(int64_t n) { return (n + kColumns - 1) / kColumns; }
int64_t sum_row_blocks(int64_t r) { return (r + kWarps * kSumRows - 1) / (kWarps * kSumRows); }
}  // namespace

int few_columns_shares(int64_t M, int64_t groups, int64_t N, int64_t K, int sm_count) {
    // blocks for two turns of the two that an SM holds, if each warp has 32 values of k
    const int64_t blocks = row_blocks(M, groups) * column_blocks(N), most = K / (32 * kWarps);
    int64_t s = 4 * (int64_t)sm_count / blocks;
    s = s > most ? most : s;
    return (int)(s < 1 ? 1 : s > 32 ? 32 : s);
}

cudaError_t launch_few_columns(const FewColumns& p, int shares, bool after_own, cudaStream_t stream) {
    if (!vec4_ok(p.A, p.lda) || !vec4_ok(p.B, p.ldb) || !vec4_ok(p.D, p.D ? p.ldd : 0) || !vec4_ok(p.C, p.ldc) ||
        (shares > 1 && !vec4_ok(p.shares, p.ldshares)))
        return cudaErrorMisalignedAddress;
    const int64_t columns = column_blocks(p.N), blocks = row_blocks(p.M, p.groups);
    if (columns > INT32_MAX || blocks > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)columns, (unsigned)blocks, (unsigned)shares);
    cudaError_t e;
    switch (block_rows(p.M, p.groups)) {
        case 1: e = launch(few_columns_kernel<1>, grid, after_own, stream, p); break;
        case 2: e = launch(few_columns_kernel<2>, grid, after_own, stream, p); break;
        case 4: e = launch(few_columns_kernel<4>, grid, after_own, stream, p); break;
        default: e = launch(few_columns_kernel<8>, grid, after_own, stream, p);
    }
    if (e != cudaSuccess || shares == 1) return e;
    const int64_t adders = ((p.N + 3) / 4 * p.M + 255) / 256;
    if (adders > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch(add_shares_kernel, dim3((unsigned)adders, 1, 1), true, stream, p, shares);
}

int few_sums_chunk(int64_t M, int64_t R, int64_t N, int sm_count) {
    // pieces for the two blocks that an SM holds if one group has all rows, of 64 rows at least
    const int64_t blocks = column_blocks(N) * sum_row_blocks(R), most = 2 * (int64_t)sm_count, pieces = (most + blocks - 1) / blocks;
    const int64_t chunk = (M + pieces - 1) / pieces;
    return (int)(chunk < 64 ? 64 : chunk);
}

cudaError_t launch_few_sums(const FewSums& p, bool after_own, cudaStream_t stream) {
    const int64_t pieces = few_sums_pieces(p.M, p.chunk);
    if (!vec4_ok(p.A, p.lda) || !vec4_ok(p.B, p.ldb) || !vec4_ok(p.C, p.ldc) || (pieces > 0 && !vec4_ok(p.pieces, p.ldpieces)))
        return cudaErrorMisalignedAddress;
    const int64_t columns = column_blocks(p.N), rows = sum_row_blocks(p.R);
    if (columns * rows > INT32_MAX || p.groups + pieces > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)(columns * rows), (unsigned)(p.groups + pieces), 1);
    return pieces == 0 ? launch(few_sums_kernel<false>, grid, after_own, stream, p, (unsigned)columns)
                       : launch(few_sums_kernel<true>, grid, after_own, stream, p, (unsigned)columns);
}

cudaError_t launch_add_pieces(const FewSums* sums, int n, cudaStream_t stream) {
    TwoSums two;
    int64_t adders = 0, pieces = 0;
    int with = 0;
    for (int i = 0; i < n; ++i) {
        const int64_t mine = few_sums_pieces(sums[i].M, sums[i].chunk);
        if (mine == 0) continue;
        two.sums[with++] = sums[i];
        const int64_t blocks = ((sums[i].N + 3) / 4 * sums[i].R + 32 * kWarps - 1) / (32 * kWarps), most = 1024 / mine + 1;
        adders = std::max(adders, std::min(blocks, most));
        pieces = std::max(pieces, mine);
    }
    if (with == 0) return cudaSuccess;
    return launch(add_pieces_kernel, dim3((unsigned)adders, (unsigned)pieces, (unsigned)with), true, stream, two);
}

}  // namespace emu
