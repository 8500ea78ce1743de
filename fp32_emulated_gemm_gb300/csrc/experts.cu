// experts.cu -- the gated blocks of a layer of experts on rows sorted by expert,
// forward and backward.
//
// Expert e has rows offsets[e] .. offsets[e+1] of X and the weights W_in[e] (the
// gate's F rows, then the up projection's) and W_out[e]:
//   [G | U] = X W_in[e]^T, H = a(G) U, Y = H W_out[e]^T;  D = [U a'(G) | a(G)]
//   dZ = [dY W_out[e] | dY W_out[e]] D, dX = dZ W_in[e],
//   dW_in[e] = dZ^T X, dW_out[e] = dY^T H over the expert's rows.
// The products run on the emulated kernel with rows or contraction in groups
// (emu_kernel.cuh): 256-row tiles that end with the expert's rows, listed on the
// device from the offsets, which never come to the host.  A few rows run on the
// CUDA cores (few_rows.cu), where each expert's weight is read once.
#include <cuda_runtime.h>

#include "activation.cuh"
#include "aligned.cuh"
#include "few_rows.h"
#include "internal.h"
#include "ptx.cuh"

namespace emu {
namespace {

constexpr int kMaxExperts = 1024, kTileRows = 256;

// The experts' row blocks (of `block` rows at most) and their bounds, from the
// offsets, which are taken as ascending and within the rows: what breaks that
// gets no rows, and nothing outside them is read or written.
// list[i] = {first row, row after the last, expert, 0}; groups[e] likewise, the
// experts of the most rows first, so that the long sums start first.
struct Lists { int4 *blocks, *groups; int* count; };

__global__ void __launch_bounds__(kMaxExperts) list_kernel(const int32_t* offsets, int E, int rows, int block, Lists out) {
    __shared__ int32_t first[kMaxExperts + 1], start[kMaxExperts + 1], sums[32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    griddep_launch_dependents();
    auto scan = [&](int v, bool largest) {  // inclusive, over the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v = largest ? max(v, up) : v + up;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        if (warp == 0) {
            int s = sums[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, s, o);
                if (lane >= o) s = largest ? max(s, up) : s + up;
            }
            sums[lane] = s;
        }
        __syncthreads();
        if (warp > 0) v = largest ? max(v, sums[warp - 1]) : v + sums[warp - 1];
        __syncthreads();
        return v;
    };
    // ends, made ascending; the first expert starts at offsets[0]
    int end = t < E ? min(max(offsets[t + 1], 0), rows) : 0;
    const int begin = min(max(offsets[0], 0), rows);
    end = max(scan(end, true), begin);
    if (t < E) first[t + 1] = end;
    if (t == 0) first[0] = begin;
    __syncthreads();
    const int r0 = t < E ? first[t] : 0, r1 = t < E ? first[t + 1] : 0, n = r1 - r0;
    if (out.groups) {
        int rank = 0;
        for (int e = 0; e < E; ++e) {
            const int m = first[e + 1] - first[e];
            rank += m > n || (m == n && e < t);
        }
        if (t < E) out.groups[rank] = make_int4(r0, r1, t, 0);
    }
    if (!out.blocks) return;
    const int tiles = (n + block - 1) / block, at = scan(tiles, false);
    if (t < E) start[t + 1] = at;
    if (t == 0) start[0] = 0;
    __syncthreads();
    const int total = start[E];
    if (t == 0) *out.count = total;
    for (int i = t; i < total; i += kMaxExperts) {
        int lo = 0, hi = E - 1;  // the expert whose blocks hold i: start[e] <= i < start[e + 1]
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (start[mid + 1] <= i) lo = mid + 1; else hi = mid;
        }
        const int b0 = first[lo] + (i - start[lo]) * block;
        out.blocks[i] = make_int4(b0, min(b0 + block, first[lo + 1]), lo, 0);
    }
}

int64_t most_blocks(int64_t rows, int E, int block) { return rows / block + (rows < E ? rows : E); }

// Buffer for the lists: the count, then the blocks, then the groups.
size_t list_floats(int64_t rows, int E, int block) { return 4 * (size_t)(1 + most_blocks(rows, E, block) + E); }
Lists lists_at(float* base, int64_t rows, int E, int block, bool blocks, bool groups) {
    int4* p = reinterpret_cast<int4*>(base);
    return {blocks ? p + 1 : nullptr, groups ? p + 1 + most_blocks(rows, E, block) : nullptr, reinterpret_cast<int*>(p)};
}
cudaError_t launch_lists(const int32_t* offsets, int E, int64_t rows, int block, const Lists& out, cudaStream_t s) {
    cudaGetLastError();
    list_kernel<<<1, kMaxExperts, 0, s>>>(offsets, E, (int)rows, block, out);
    return cudaGetLastError();
}

// Few rows for each expert: the CUDA cores, on which the weights of the experts
// that have rows are read once.
bool few(int64_t rows, int E) { return rows <= 4 * (int64_t)E; }
int few_block_rows(int64_t rows, int E) { return 4 * rows <= E ? 1 : rows <= E ? 2 : rows <= 3 * (int64_t)E ? 4 : 8; }

bool size_ok(int64_t v) { return v <= INT32_MAX - 256; }

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" {

emu_status_t emu_expert_ffn_fwd(emu_mode_t mode, emu_act_t act, int64_t rows, int E, int64_t K, int64_t F, int64_t N,
                                const float* X, int64_t ldx, const int32_t* offsets, const float* W_in, int64_t ldwi,
                                const float* W_out, int64_t ldwo, float* D, int64_t ldd, float* H, int64_t ldh, float* Y,
                                int64_t ldy, emu_stream_t stream) {
    if (act < EMU_ACT_NONE || act > EMU_ACT_SILU || rows < 0 || E < 1 || K < 1 || F < 1 || N < 1)
        return EMU_STATUS_INVALID_VALUE;
    if (!fused_mode(mode) || E > kMaxExperts || !size_ok(rows) || !size_ok(K) || !size_ok(2 * F) || !size_ok(N) ||
        !size_ok(E * 2 * F) || !size_ok(E * N))
        return EMU_STATUS_NOT_SUPPORTED;
    if (rows == 0) return EMU_STATUS_SUCCESS;
    if (!X || !offsets || !W_in || !W_out || !H || !Y || ldx < K || ldwi < K || ldwo < F || ldh < F || ldy < N ||
        (D && ldd < 2 * F))
        return EMU_STATUS_INVALID_VALUE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    DeviceCtx dev;
    float* scratch = nullptr;
    if (few(rows, E)) {
        const int block = few_block_rows(rows, E);
        EMU_TRY(current_device(&dev));
        EMU_TRY(reduce_scratch(dev.id, s, list_floats(rows, E, block), &scratch));
        const Lists l = lists_at(scratch, rows, E, block, true, false);
        EMU_TRY(launched(launch_lists(offsets, E, rows, block, l, s)));
        FewRows p{(int)rows, F, K, X, ldx, W_in, ldwi, nullptr, nullptr, 0, D, ldd, H, ldh, act_params(act)};
        p.list = l.blocks;
        p.count = l.count;
        p.blocks = (int)most_blocks(rows, E, block);
        EMU_TRY(launched(launch_few_rows_grouped(p, block, true, dev.sm_count, s)));
        p.N = N; p.K = F; p.X = H; p.ldx = ldh; p.W = W_out; p.ldw = ldwo; p.D = nullptr; p.Y = Y; p.ldy = ldy;
        p.act = act_params(ACT_NONE);
        return launched(launch_few_rows_grouped(p, block, false, dev.sm_count, s));
    }
    if (D && !vec4_ok(D, ldd)) return EMU_STATUS_NOT_SUPPORTED;
    Aligned al;
    al.add(X, ldx, rows, K);
    al.add(W_in, ldwi, E * 2 * F, K);
    al.add(W_out, ldwo, E * N, F);
    Lists l{};
    auto products = [&](Until until) {
        const Fused f{FUSED_GATED, act, nullptr, 0, D, ldd, nullptr};
        GroupedGemm g{false, E, false, rows, 0, F, K, X, ldx, W_in, ldwi, H, ldh, &f, l.blocks, l.count};
        EMU_TRY(gemm_grouped(mode, g, s, until));
        g = {false, E, false, rows, 0, N, F, H, ldh, W_out, ldwo, Y, ldy, nullptr, l.blocks, l.count};
        return gemm_grouped(mode, g, s, until);
    };
    al.stand_in();
    EMU_TRY(products(UNTIL_CHECKED));
    EMU_TRY(current_device(&dev));
    EMU_TRY(al.reserve(s));
    EMU_TRY(reduce_scratch(dev.id, s, list_floats(rows, E, kTileRows), &scratch));
    l = lists_at(scratch, rows, E, kTileRows, true, false);
    EMU_TRY(launched(al.launch(s)));
    EMU_TRY(launched(launch_lists(offsets, E, rows, kTileRows, l, s)));
    return products(UNTIL_LAUNCHED);
}

emu_status_t emu_expert_ffn_bwd(emu_mode_t mode, int64_t rows, int E, int64_t K, int64_t F, int64_t N, const float* dY,
                                int64_t lddy, const float* X, int64_t ldx, const int32_t* offsets, const float* W_in,
                                int64_t ldwi, const float* W_out, int64_t ldwo, const float* D, int64_t ldd, const float* H,
                                int64_t ldh, float* dZ, int64_t lddz, float* dX, int64_t lddx, float* dW_in, int64_t lddwi,
                                float* dW_out, int64_t lddwo, emu_stream_t stream) {
    if (rows < 0 || E < 1 || K < 1 || F < 1 || N < 1) return EMU_STATUS_INVALID_VALUE;
    if (!fused_mode(mode) || E > kMaxExperts || !size_ok(rows) || !size_ok(K) || !size_ok(2 * F) || !size_ok(N) ||
        !size_ok(E * 2 * F) || !size_ok(E * N))
        return EMU_STATUS_NOT_SUPPORTED;
    if ((dW_in && lddwi < K) || (dW_out && lddwo < F)) return EMU_STATUS_INVALID_VALUE;
    const bool inner = dX || dW_in;
    if (!inner && !dW_out) return EMU_STATUS_SUCCESS;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    DeviceCtx dev;
    if (rows == 0) {  // empty sums
        EMU_TRY(current_device(&dev));
        if (dW_in) EMU_TRY(launched(cudaMemset2DAsync(dW_in, lddwi * sizeof(float), 0, K * sizeof(float), E * 2 * F, s)));
        if (dW_out) EMU_TRY(launched(cudaMemset2DAsync(dW_out, lddwo * sizeof(float), 0, F * sizeof(float), E * N, s)));
        return EMU_STATUS_SUCCESS;
    }
    if (!dY || !offsets || lddy < N) return EMU_STATUS_INVALID_VALUE;
    if (inner && (!W_out || !D || !dZ || ldwo < F || ldd < 2 * F || lddz < 2 * F)) return EMU_STATUS_INVALID_VALUE;
    if (dX && (!W_in || ldwi < K || lddx < K)) return EMU_STATUS_INVALID_VALUE;
    if (dW_in && (!X || ldx < K)) return EMU_STATUS_INVALID_VALUE;
    if (dW_out && (!H || ldh < F)) return EMU_STATUS_INVALID_VALUE;
    Aligned al;
    al.add(dY, lddy, rows, N);
    if (inner) {
        al.add(W_out, ldwo, E * N, F);
        al.add(D, ldd, rows, 2 * F);
    }
    if (dX) al.add(W_in, ldwi, E * 2 * F, K);
    if (dW_in) al.add(X, ldx, rows, K);
    if (dW_out) al.add(H, ldh, rows, F);
    Lists l{};
    auto products = [&](Until until) {
        if (inner) {
            const Fused f{FUSED_GATED_BWD, ACT_NONE, nullptr, 0, const_cast<float*>(D), ldd, nullptr};
            const GroupedGemm g{false, E, true, rows, 0, F, N, dY, lddy, W_out, ldwo, dZ, lddz, &f, l.blocks, l.count};
            EMU_TRY(gemm_grouped(mode, g, s, until));
        }
        if (dW_out) {
            const GroupedGemm g{true, E, true, rows, N, F, 0, dY, lddy, H, ldh, dW_out, lddwo, nullptr, l.groups, nullptr};
            EMU_TRY(gemm_grouped(mode, g, s, until));
        }
        if (dX) {
            const GroupedGemm g{false, E, true, rows, 0, K, 2 * F, dZ, lddz, W_in, ldwi, dX, lddx, nullptr, l.blocks, l.count};
            EMU_TRY(gemm_grouped(mode, g, s, until));
        }
        if (dW_in) {
            const GroupedGemm g{true, E, true, rows, 2 * F, K, 0, dZ, lddz, X, ldx, dW_in, lddwi, nullptr, l.groups, nullptr};
            EMU_TRY(gemm_grouped(mode, g, s, until));
        }
        return EMU_STATUS_SUCCESS;
    };
    al.stand_in();
    EMU_TRY(products(UNTIL_CHECKED));
    EMU_TRY(current_device(&dev));
    EMU_TRY(al.reserve(s));
    float* scratch = nullptr;
    EMU_TRY(reduce_scratch(dev.id, s, list_floats(rows, E, kTileRows), &scratch));
    l = lists_at(scratch, rows, E, kTileRows, inner, dW_in || dW_out);
    EMU_TRY(launched(al.launch(s)));
    EMU_TRY(launched(launch_lists(offsets, E, rows, kTileRows, l, s)));
    return products(UNTIL_LAUNCHED);
}

}  // extern "C"
