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
//
// Both modes run as BF16x9, which is within TF32x3's bound too: TF32x3 without an
// operand split ahead is slower (12288 rows on 8 experts, K = 256, F = 1024, the six
// products of a training step: BF16x9 105, 48, 93, 50, 74, 80 us, TF32x3 122, 58,
// 102, 60, 98, 98), and the sums over an expert's rows, which start anywhere, could
// not load split rows (a copy starts on 16 bytes).
#include <cuda_runtime.h>

#include "activation.cuh"
#include "aligned.cuh"
#include "emu_kernel.cuh"
#include "few_rows.h"
#include "internal.h"

namespace emu {
namespace {

constexpr int kMaxExperts = 1024, kTileRows = 256;

// The experts' row tiles (256 rows at most) and their bounds, from the
// offsets, which are taken as ascending and within the rows: what breaks that
// gets no rows, and nothing outside them is read or written.
// blocks[i] = {first row, row after the last, expert, 0}; groups[e] likewise, the
// experts of the most rows first, so that whole tiles taken in turn leave the
// short ones for the end.
struct Lists { int4 *blocks, *groups; };

// The walks of the CTA pairs of up to four products (GroupWalk).
constexpr int kMaxProducts = 4;
struct Walks {
    int n, pairs;
    GroupWalk* out;               // n x pairs
    bool sum[kMaxProducts];
    GroupedTiles tiles[kMaxProducts];
};

// A product's tiles in turn (0), or equal runs of its stages, on how many pairs: what
// is predicted faster for the longest of them, in stages.  A tile's stores cost 3,
// publishing a piece 1.5 and adding one 2.  Fewer runs than pairs where a tile would
// be cut into many pieces, which one pair adds up.
__device__ int cut_tiles(bool sum, GroupedTiles tiles, int entries, const int4* groups, int64_t total, int pairs) {
    const int64_t n = (int64_t)entries * tiles.per, waves = (n + pairs - 1) / pairs;
    if (n == 0) return 0;
    const int shortest = (int)((total + pairs - 1) / pairs);  // a run on all pairs
    int longest = tiles.stages;
    float whole = 0.f;
    if (sum) {
        longest = group_stages(groups[0].y - groups[0].x);
        // (the first pair's tiles are the longest of each wave)
        for (int64_t w = 0; w < waves && whole <= 4.f * (shortest + longest) + 100.f; ++w) {
            const int4 g = groups[w * pairs / tiles.per];
            whole += group_stages(g.y - g.x) + 3.f;
        }
    } else {
        whole = (float)waves * (longest + 3.f);
    }
    float best = whole / 1.03f;
    int runs = 0;
    for (int pieces = 0; pieces <= 8; ++pieces) {
        const int run = pieces == 0 ? shortest : (longest + pieces - 1) / pieces;
        if (run < shortest || run < 2) continue;
        const int r = (int)((total + run - 1) / run);
        const float cost = run + 3.f * (float)((n + r - 1) / r) + 1.5f + 2.f * ((longest + run - 1) / run);
        if (cost < best) {
            best = cost;
            runs = r;
        }
    }
    return runs;
}

__global__ void __launch_bounds__(kMaxExperts)
list_kernel(const int32_t* offsets, int E, int rows, Lists out, const __grid_constant__ Walks walks) {
    __shared__ int32_t first[kMaxExperts + 1], start[kMaxExperts + 1], sums[32];
    __shared__ int4 sorted[kMaxExperts];
    __shared__ int cut[kMaxProducts];
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
    int blocks_total = 0;
    if (out.blocks) {
        const int tiles = (n + kTileRows - 1) / kTileRows, at = scan(tiles, false);
        if (t < E) start[t + 1] = at;
        if (t == 0) start[0] = 0;
        __syncthreads();
        blocks_total = start[E];
        for (int i = t; i < blocks_total; i += kMaxExperts) {
            int lo = 0, hi = E - 1;  // the expert whose blocks hold i: start[e] <= i < start[e + 1]
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (start[mid + 1] <= i) lo = mid + 1; else hi = mid;
            }
            const int b0 = first[lo] + (i - start[lo]) * kTileRows;
            out.blocks[i] = make_int4(b0, min(b0 + kTileRows, first[lo + 1]), lo, 0);
        }
        __syncthreads();
    }
    if (out.groups) {
        int rank = 0;
        for (int e = 0; e < E; ++e) {
            const int m = first[e + 1] - first[e];
            rank += m > n || (m == n && e < t);
        }
        if (t < E) out.groups[rank] = sorted[rank] = make_int4(r0, r1, t, 0);
        __syncthreads();
        // start[i]: stages of the first i of the sorted experts
        const int at = scan(t < E ? group_stages(sorted[t].y - sorted[t].x) : 0, false);
        if (t < E) start[t + 1] = at;
        if (t == 0) start[0] = 0;
        __syncthreads();
    }
    auto entries = [&](int k) { return walks.sum[k] ? E : blocks_total; };
    auto total = [&](int k) {
        const int64_t per = walks.tiles[k].per;
        return walks.sum[k] ? per * start[E] : per * blocks_total * walks.tiles[k].stages;
    };
    if (t < walks.n)
        cut[t] = cut_tiles(walks.sum[t], walks.tiles[t], entries(t), sorted, total(t), walks.pairs);
    __syncthreads();
    for (int i = t; i < walks.n * walks.pairs; i += kMaxExperts) {
        const int k = i / walks.pairs, pair = i - k * walks.pairs;
        const GroupedTiles tiles = walks.tiles[k];
        GroupWalk w{};
        w.hi = INT32_MAX;
        if (!cut[k]) {
            w.first = pair;
            w.last = entries(k) * tiles.per;
            w.step = walks.pairs;
        } else if (pair < cut[k]) {
            const int64_t U = total(k);
            const int runs = cut[k], run = runs - 1 - pair;
            const int64_t s = run * U / runs, e = (run + 1) * U / runs;  // (a run has two stages or more)
            // the tile at position x, its first position and its stages
            auto tile_at = [&](int64_t x, int64_t& base, int& stages) {
                if (!walks.sum[k]) {
                    stages = tiles.stages;
                    const int64_t tile = x / stages;
                    base = tile * stages;
                    return (int)tile;
                }
                int lo = 0, hi = E - 1;
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if ((int64_t)start[mid + 1] * tiles.per <= x) lo = mid + 1; else hi = mid;
                }
                stages = start[lo + 1] - start[lo];
                base = (int64_t)start[lo] * tiles.per;
                const int64_t j = (x - base) / stages;
                base += j * stages;
                return lo * tiles.per + (int)j;
            };
            int64_t base;
            int stages;
            w.first = tile_at(s, base, stages);
            w.lo = (int)(s - base);
            w.last = tile_at(e - 1, base, stages) + 1;
            w.hi = (int)(e - base);
            w.step = 1;
            // the next runs that start within the last tile
            for (int r = run + 1; r < runs && r * U / runs < base + stages; ++r) ++w.others;
        }
        walks.out[i] = w;
    }
}

int64_t most_blocks(int64_t rows, int E) { return rows / kTileRows + (rows < E ? rows : E); }

// Buffer for the lists: the blocks, the groups, the walks.
size_t list_floats(int64_t rows, int E, int walks) {
    return 4 * (size_t)(most_blocks(rows, E) + E) + walks * (sizeof(GroupWalk) / sizeof(float));
}
struct Listed {
    Lists lists;
    GroupWalk* walks;
};
Listed lists_at(float* base, int64_t rows, int E, bool blocks, bool groups) {
    int4 *p = reinterpret_cast<int4*>(base), *g = p + most_blocks(rows, E);
    return {{blocks ? p : nullptr, groups ? g : nullptr}, reinterpret_cast<GroupWalk*>(g + E)};
}
cudaError_t launch_lists(const int32_t* offsets, int E, int64_t rows, const Lists& out, const Walks& walks, cudaStream_t s) {
    cudaGetLastError();
    list_kernel<<<1, kMaxExperts, 0, s>>>(offsets, E, (int)rows, out, walks);
    return cudaGetLastError();
}

// Few rows for each expert: the CUDA cores, on which the weights of the experts
// that have rows are read once.
bool few(int64_t rows, int E) { return rows <= 8 * (int64_t)E; }

bool size_ok(int64_t v) { return v <= INT32_MAX - 256; }

// A call's grouped products, one after the other, with one launch for the lists and
// walks of all of them.
struct Products {
    int64_t rows;
    int E, n = 0;
    bool blocks = false, groups = false;
    GroupedGemm g[kMaxProducts];

    Products(int64_t r, int e) : rows(r), E(e) {}
    void add(const GroupedGemm& p) {
        (p.sum ? groups : blocks) = true;
        g[n++] = p;
    }
    emu_status_t run(cudaStream_t s, Until until) const {
        for (int i = 0; i < n; ++i) EMU_TRY(gemm_grouped(g[i], s, until));
        return EMU_STATUS_SUCCESS;
    }
    emu_status_t launch(const int32_t* offsets, const Listed& l, int pairs, cudaStream_t s) {
        Walks w{n, pairs, l.walks, {}, {}};
        for (int i = 0; i < n; ++i) {
            w.sum[i] = g[i].sum;
            w.tiles[i] = grouped_tiles(g[i]);
            g[i].list = g[i].sum ? l.lists.groups : l.lists.blocks;
            g[i].walks = l.walks + (int64_t)i * pairs;
        }
        EMU_TRY(launched(launch_lists(offsets, E, rows, l.lists, w, s)));
        return run(s, UNTIL_LAUNCHED);
    }
};

// In steps: the arguments' checks, the buffers, then the copies of odd operands,
// the lists and the products.  make() gives the products with the operands'
// addresses as they are at the time.
template <class F> emu_status_t run_products(Aligned& al, F make, const int32_t* offsets, cudaStream_t s) {
    al.stand_in();
    Products q = make();
    EMU_TRY(q.run(s, UNTIL_CHECKED));
    DeviceCtx dev;
    EMU_TRY(current_device(&dev));
    EMU_TRY(al.reserve(s));
    EMU_TRY(q.run(s, UNTIL_RESERVED));
    int pairs = 0;
    EMU_TRY(grouped_pairs(&pairs));
    float* scratch = nullptr;
    EMU_TRY(reduce_scratch(dev.id, s, list_floats(q.rows, q.E, q.n * pairs), &scratch));
    EMU_TRY(launched(al.launch(s)));
    q = make();
    return q.launch(offsets, lists_at(scratch, q.rows, q.E, q.blocks, q.groups), pairs, s);
}

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
    if (few(rows, E)) {
        EMU_TRY(current_device(&dev));
        FewRows p{(int)rows, F, K, X, ldx, W_in, ldwi, nullptr, nullptr, 0, D, ldd, H, ldh, act_params(act)};
        p.offsets = offsets;
        p.groups = E;
        EMU_TRY(launched(launch_few_rows_grouped(p, true, false, dev.sm_count, s)));
        p.N = N; p.K = F; p.X = H; p.ldx = ldh; p.W = W_out; p.ldw = ldwo; p.D = nullptr; p.Y = Y; p.ldy = ldy;
        p.act = act_params(ACT_NONE);
        return launched(launch_few_rows_grouped(p, false, true, dev.sm_count, s));
    }
    if (D && !vec4_ok(D, ldd)) return EMU_STATUS_NOT_SUPPORTED;
    Aligned al;
    al.add(X, ldx, rows, K);
    al.add(W_in, ldwi, E * 2 * F, K);
    al.add(W_out, ldwo, E * N, F);
    const Fused f{FUSED_GATED, act, nullptr, 0, D, ldd, nullptr};
    auto products = [&] {
        Products q(rows, E);
        q.add({false, E, false, rows, 0, F, K, X, ldx, W_in, ldwi, H, ldh, &f});
        q.add({false, E, false, rows, 0, N, F, H, ldh, W_out, ldwo, Y, ldy});
        return q;
    };
    return run_products(al, products, offsets, s);
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
    Fused f{};
    auto products = [&] {
        f = {FUSED_GATED_BWD, ACT_NONE, nullptr, 0, const_cast<float*>(D), ldd, nullptr};
        Products q(rows, E);
        if (inner) q.add({false, E, true, rows, 0, F, N, dY, lddy, W_out, ldwo, dZ, lddz, &f});
        if (dW_out) q.add({true, E, true, rows, N, F, 0, dY, lddy, H, ldh, dW_out, lddwo});
        if (dX) q.add({false, E, true, rows, 0, K, 2 * F, dZ, lddz, W_in, ldwi, dX, lddx});
        if (dW_in) q.add({true, E, true, rows, 2 * F, K, 0, dZ, lddz, X, ldx, dW_in, lddwi});
        return q;
    };
    return run_products(al, products, offsets, s);
}

}  // extern "C"
