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
// device from the offsets, which never come to the host.  Backward, the products
// that do not depend on one another share a launch (dZ and dW_out, dX and dW_in).
// A few rows run on the CUDA cores (few_rows.cu, few_tiles.cu, few_rows_bwd.cu), where
// each expert's weight is read once.
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
#include "few_rows_bwd.h"
#include "few_tiles.h"
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

// The walks of the CTA pairs of up to two launches (GroupWalk), each of a product
// over rows, a sum over the experts' rows, or both side by side.
constexpr int kMaxLaunches = 2, kMaxPairs = 1024;
struct Walks {
    int n, pairs;
    GroupWalk* out;                  // n x pairs
    int sum_store;                   // a sum's GroupedTiles::store
    GroupedTiles tiles[kMaxLaunches][2];  // rows, sum; per 0: there is none
};

// A tile costs its k-stages and, for its stores, `tiles.store` more: its length.
__device__ __forceinline__ int tile_length(const GroupedTiles& tiles, const int4& group) {
    return tiles.store + (tiles.sum ? group_stages(group.y - group.x) : tiles.stages);
}

// How a product's tiles go to `pairs` pairs: in turn (runs 0), or cut into runs of
// equal length; and the longest pair's time, in stages.  Publishing a piece costs 1.5
// and adding one 2.  Fewer runs than pairs where a tile would be cut into many
// pieces, which one pair adds up.  (All in FP32: integer divisions in a chain would
// cost this kernel more than they are worth.)
struct Cut {
    float cost;
    int runs;
};
__device__ Cut cut_tiles(const GroupedTiles& tiles, int entries, const int4* groups, int64_t total, int pairs) {
    const int64_t n = (int64_t)entries * tiles.per;
    if (n == 0 || pairs == 0) return {n == 0 ? 0.f : 1e30f, 0};
    const float waves = ceilf(__fdividef((float)n, (float)pairs)), shortest = ceilf(__fdividef((float)total, (float)pairs));  // a run on all pairs
    const float longest = (float)tile_length(tiles, groups[0]);  // (sorted)
    float whole = waves * longest;
    if (tiles.sum) {
        whole = shortest + 0.5f * longest;
        if (waves <= 8.f) {  // the first pair's tiles are the longest of each wave
            whole = 0.f;
            for (int w = 0; w < (int)waves; ++w)
                whole += (float)tile_length(tiles, groups[min(w * pairs / tiles.per, entries - 1)]);
        }
    }
    Cut best{whole, 0};
    float best_run = 0.f;
#pragma unroll 1
    for (int pieces = 0; pieces <= 8; ++pieces) {
        const float run = pieces == 0 ? shortest : ceilf(__fdividef(longest, (float)pieces));
        if (run < shortest || run < 2.f) continue;
        const float cost = run + 1.5f + 2.f * ceilf(__fdividef(longest, run));
        if (1.03f * cost < best.cost) {
            best.cost = cost;
            best_run = run;
        }
    }
    if (best_run > 0.f) best.runs = (int)fminf(ceilf((float)total / best_run), (float)pairs);
    return best;
}

// Threads: at least one an expert (all sums over the experts are one scan) and 256.
__global__ void __launch_bounds__(kMaxExperts)
list_kernel(const int32_t* offsets, int E, int rows, Lists out, const __grid_constant__ Walks walks) {
    __shared__ int32_t first[kMaxExperts + 1], start[kMaxExperts + 1], sums[32];
    __shared__ int4 sorted[kMaxExperts];
    __shared__ int split[kMaxLaunches], runs[kMaxLaunches][2];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    griddep_launch_dependents();
    griddep_wait();  // the offsets are another kernel's, and the last call's products may still read the lists
    auto scan = [&](int v, bool largest) {  // inclusive, over the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v = largest ? max(v, up) : v + up;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        if (warp == 0) {
            int s = lane < (int)blockDim.x / 32 ? sums[lane] : 0;
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
        for (int i = t; i < blocks_total; i += (int)blockDim.x) {
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
        // start[i]: lengths of a tile of each of the first i of the sorted experts (all
        // sums' stores cost the same)
        const int at = scan(t < E ? group_stages(sorted[t].y - sorted[t].x) + walks.sum_store : 0, false);
        if (t < E) start[t + 1] = at;
        if (t == 0) start[0] = 0;
        __syncthreads();
    }
    auto entries = [&](const GroupedTiles& k) { return k.sum ? E : blocks_total; };
    auto total = [&](const GroupedTiles& k) {
        return k.sum ? (int64_t)k.per * start[E] : (int64_t)k.per * blocks_total * (k.stages + k.store);
    };
    // a launch's pairs: the rows' product has the first `split`; of 32 splits, a lane
    // each, the one whose longer side is the shortest
    if (warp < walks.n) {
        const GroupedTiles &r = walks.tiles[warp][0], &s = walks.tiles[warp][1];
        const int pairs = walks.pairs, first_pairs = s.per == 0 ? pairs : r.per == 0 ? 0 : 1 + (pairs - 2) * lane / 31;
        Cut a{0.f, 0}, b{0.f, 0};
        if (r.per) a = cut_tiles(r, entries(r), sorted, total(r), first_pairs);
        if (s.per) b = cut_tiles(s, entries(s), sorted, total(s), pairs - first_pairs);
        const float cost = fmaxf(a.cost, b.cost);
        float least = cost;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
        if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, cost == least)) - 1) {
            split[warp] = first_pairs;
            runs[warp][0] = a.runs;
            runs[warp][1] = b.runs;
        }
    }
    __syncthreads();
    for (int i = t; i < walks.n * walks.pairs; i += (int)blockDim.x) {
        const int k = i / walks.pairs, cid = i - k * walks.pairs, second = cid >= split[k];
        const GroupedTiles tiles = walks.tiles[k][second];
        const int pair = cid - (second ? split[k] : 0), pairs = second ? walks.pairs - split[k] : split[k];
        const int cut = runs[k][second], run = cut - 1 - pair;
        GroupWalk w{};
        w.hi = INT32_MAX;
        w.second = second;
        w.step = 1;
        if (cut == 0) {
            w.first = pair;
            w.last = entries(tiles) * tiles.per;
            w.step = pairs;
        } else if (run >= 0) {
            const int64_t U = total(tiles);
            // where run r starts, r U / cut (a run has a length of two or more)
            auto start_of = [&](int r) {
                return U <= INT32_MAX / kMaxPairs ? (int64_t)((uint32_t)r * (uint32_t)U / (uint32_t)cut) : r * U / cut;
            };
            // the tile that length x falls into, its end, and the stage: the first
            // `store` of a tile's length are its stores, and a run that starts within
            // them has the whole tile
            struct At { int tile, stage; int64_t end; };
            auto at = [&](int64_t x) {
                int length = tiles.stages + tiles.store, first_tile = 0;
                int64_t base = 0;
                if (tiles.sum) {
                    int lo = 0, hi = E - 1;
                    while (lo < hi) {
                        const int mid = (lo + hi) / 2;
                        if ((int64_t)start[mid + 1] * tiles.per <= x) lo = mid + 1; else hi = mid;
                    }
                    length = start[lo + 1] - start[lo];
                    base = (int64_t)start[lo] * tiles.per;
                    first_tile = lo * tiles.per;
                }
                const int64_t j = x - base <= UINT32_MAX ? (uint32_t)(x - base) / (uint32_t)length : (x - base) / length;
                base += j * length;
                return At{first_tile + (int)j, max((int)(x - base) - tiles.store, 0), base + length};
            };
            const At s = at(start_of(run));
            w.first = s.tile;
            w.lo = s.stage;
            if (run + 1 == cut) {
                w.last = entries(tiles) * tiles.per;
            } else {
                const At e = at(start_of(run + 1));
                w.last = e.tile;
                if (e.stage > 0 && !(e.tile == s.tile && e.stage <= s.stage)) {
                    w.last = e.tile + 1;
                    w.hi = e.stage;
                    // the next runs that start within the last tile
                    for (int r = run + 1; r < cut && start_of(r) < e.end; ++r) ++w.others;
                }
            }
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(E <= 256 ? 256 : kMaxExperts, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, list_kernel, offsets, E, (int)rows, out, walks);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

// A forward pass in one of three forms: on the CUDA cores, where the weights of the
// experts that have rows are read once for eight rows (few_rows.cu) or for 16 or 32
// through shared memory (few_tiles.cu), or in 256-row tiles: the one of the least
// predicted time, in us.  The first one's is the rows' share of each step of 128 of
// each lot of weight rows and of the lots' sums, and the weights' traffic where L2 does
// not hold them; the second's its FMAs, an expert's last rows rounded up; the tiles'
// their lengths (k-stages and stores) over the CTA pairs, or the longest's own, cut in
// pieces.  Measured, first / second / tiles: 8 experts, K = 1024, F = 4096, 32 rows 89 /
// 120 / 251 us, 128 rows 196 / 141 / 253, 512 rows 688 / 403 / 261; 8 experts, K = 256, F
// = 1024, 256 rows 33 / 32 / 59, 512 rows 58 / 35 / 60, 2048 rows - / 93 / 69; 64 experts,
// K = 512, F = 1024, 256 rows 87 / 101 / 218, 512 rows 125 / 117 / 232, 1024 rows 215 / 149
// / 257; 16 experts, K = F = 1024, 64 rows 51 / 64 / 147, 256 rows 110 / 85 / 150, 1024 rows
// 321 / 208 / 152; 2 experts, K = F = 64, 256 rows 6 / 12 / 33, 16384 rows 74 / - / 35.
constexpr int64_t kFewRowsMost = 32768;
constexpr int kPairs = 76;
constexpr double kL2Weights = 25e6;  // weights that stay in L2 beside the rest
enum Form { FORM_ROWS, FORM_SHARED, FORM_TILES };
Form form_of(int64_t rows, int E, int64_t K, int64_t F, int64_t N, int pairs, bool shared_fits) {
    if (rows > kFewRowsMost) return FORM_TILES;
    auto over = [](int64_t n, int64_t d) { return (double)((n + d - 1) / d); };
    const double T = (double)rows, used = rows < E ? T : (double)E, W = (double)F * (2.0 * K + N);
    const double lots = 0.5 * F + 0.25 * N, steps = 0.5 * F * over(K, 128) + 0.25 * N * over(F, 128);
    double cores = 4.0 + T * (3.74e-5 * steps + 3.4e-5 * lots);
    if (E * W > kL2Weights) cores += (T / 8 + 0.5 * used) * W * 4 / 8e6;
    const double shared = shared_fits ? 9.0 + (T + 10 * used) * W / 17.5e6 : 1e30;
    const double half = T / 256 + 0.5 * E, tiles = used > half ? used : half;
    auto product = [&](double columns, double stages) {
        const double length = stages + 3, share = tiles * columns * length / pairs, least = length < 12 ? length : 12;
        return 1.44 * (share > least ? share : least);
    };
    const double tiled = 22.0 + product(over(F, 128), over(K, 32)) + product(over(N, 256), over(F, 32));
    return cores <= tiled && cores <= shared ? FORM_ROWS : shared <= tiled ? FORM_SHARED : FORM_TILES;
}
// Likewise for a backward pass (few_rows_bwd.cu): the weights read and their gradients
// written, and the rows' products or, for small weights, the sums' way through an
// expert's rows; the tiles' two launches, whose length dZ's stores and a sum's few
// stages make.  Measured, CUDA cores / tiles: 8 experts, K = 256, F = 1024, 8 rows 24 / 81
// us, 128 rows 56 / 87, 512 rows 134 / 94; 64 experts, K = 512, F = 1024, 64 rows 206 /
// 309, 512 rows 415 / 456, 1024 rows 634 / 498; 8 experts, K = 1024, F = 4096, 2 rows 132 /
// 212, 32 rows 318 / 383, 128 rows 604 / 445; 2 experts, K = F = 64, 64 rows 32 / 46, 128
// rows 54 / 48.  (Chunks of an expert's rows, for the sums of more than 64, cost 1 to 5%
// of these and hold the form's time where one expert has most rows: few_rows_bwd.cu.)
bool few_bwd(int64_t rows, int E, int64_t K, int64_t F, int64_t N, int pairs) {
    if (rows > kFewRowsMost) return false;
    auto over = [](int64_t n, int64_t d) { return (double)((n + d - 1) / d); };
    const double T = (double)rows, used = rows < E ? T : (double)E, W = (double)F * (2.0 * K + N);
    const double product = 2.4e-7 * W, latency = 1.1 / E;
    const double cores = 1.15 * (12.0 + (E + used) * W * 4 / 5.5e6 + T * (product > latency ? product : latency));
    const double half = T / 256 + 0.5 * E, tiles = used > half ? used : half;
    const double stages = T / E / 32 < 1 ? 1.0 : T / E / 32;  // a sum's
    auto launch = [&](double columns, double length, double sums) {
        const double share = (tiles * columns * length + E * sums * (stages + 3)) / pairs, least = length < 16 ? length : 16;
        return 1.44 * (share > least ? share : least);
    };
    return cores <= 28.0 + launch(over(F, 256), over(N, 32) + 14, over(N, 256) * over(F, 256)) +
                        launch(over(K, 256), over(2 * F, 32) + 3, over(2 * F, 256) * over(K, 256));
}
// Lots of weight rows (two of each half, or four) that make the streaming form the
// faster one (few_rows.cu).
bool many_lots(int64_t rows, int64_t F, int64_t N) { return rows * (F / 2 + N / 4) >= 8192; }

bool size_ok(int64_t v) { return v <= INT32_MAX - 256; }
// (each size before its products, which would overflow)
bool sizes_ok(int64_t rows, int E, int64_t K, int64_t F, int64_t N) {
    return E <= kMaxExperts && size_ok(rows) && size_ok(K) && size_ok(F) && size_ok(N) && size_ok(E * 2 * F) && size_ok(E * N);
}

// A call's grouped products, a launch or two, with one kernel for the lists and
// walks of all of them.
struct Products {
    int64_t rows;
    int E, n = 0;
    struct Launch {
        bool has[2] = {false, false};
        GroupedGemm g[2];  // over rows, a sum
        const GroupedGemm* product(int i) const { return has[i] ? &g[i] : nullptr; }
    } launches[kMaxLaunches];

    Products(int64_t r, int e) : rows(r), E(e) {}
    void begin() { ++n; }  // a launch; what follows is its products
    void add(const GroupedGemm& p) {
        launches[n - 1].has[p.sum] = true;
        launches[n - 1].g[p.sum] = p;
    }
    emu_status_t run(cudaStream_t s, Until until) const {
        for (int i = 0; i < n; ++i)
            EMU_TRY(gemm_grouped(launches[i].product(0), launches[i].product(1), s, until));
        return EMU_STATUS_SUCCESS;
    }
    emu_status_t launch(const int32_t* offsets, float* scratch, int pairs, cudaStream_t s) {
        const Listed l = lists_at(scratch, rows, E, launches[0].has[0] || launches[n - 1].has[0],
                                  launches[0].has[1] || launches[n - 1].has[1]);
        Walks w{n, pairs, l.walks, 0, {}};
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < 2; ++j)
                if (launches[i].has[j]) {
                    w.tiles[i][j] = grouped_tiles(launches[i].g[j]);
                    if (j) w.sum_store = w.tiles[i][j].store;
                    launches[i].g[j].list = j ? l.lists.groups : l.lists.blocks;
                    launches[i].g[j].walks = l.walks + (int64_t)i * pairs;
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
    if (pairs < 2 || pairs > kMaxPairs) return EMU_STATUS_NOT_SUPPORTED;  // (two products share them)
    float* scratch = nullptr;
    EMU_TRY(reduce_scratch(dev.id, s, list_floats(q.rows, q.E, q.n * pairs), &scratch));
    EMU_TRY(launched(al.launch(s)));
    q = make();
    return q.launch(offsets, scratch, pairs, s);
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
    if (!fused_mode(mode) || !sizes_ok(rows, E, K, F, N)) return EMU_STATUS_NOT_SUPPORTED;
    if (rows == 0) return EMU_STATUS_SUCCESS;
    if (!X || !offsets || !W_in || !W_out || !H || !Y || ldx < K || ldwi < K || ldwo < F || ldh < F || ldy < N ||
        (D && ldd < 2 * F))
        return EMU_STATUS_INVALID_VALUE;
    if (!vec4_ok(H, ldh) || !vec4_ok(Y, ldy) || (D && !vec4_ok(D, ldd))) return EMU_STATUS_NOT_SUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamLock lock(s);
    DeviceCtx dev;
    FewRows in{(int)rows, F, K, X, ldx, W_in, ldwi, nullptr, nullptr, 0, D, ldd, H, ldh, act_params(act)};
    in.offsets = offsets;
    in.groups = E;
    FewRows out{(int)rows, N, F, H, ldh, W_out, ldwo, nullptr, nullptr, 0, nullptr, 0, Y, ldy, act_params(ACT_NONE)};
    out.offsets = offsets;
    out.groups = E;
    const Form form = form_of(rows, E, K, F, N, kPairs, few_tiles_fit(in) && few_tiles_fit(out));
    if (form != FORM_TILES) EMU_TRY(current_device(&dev));
    if (form == FORM_ROWS) {
        const bool streaming = many_lots(rows, F, N);
        EMU_TRY(launched(launch_few_rows_grouped(in, true, streaming, false, dev.sm_count, s)));
        return launched(launch_few_rows_grouped(out, false, streaming, true, dev.sm_count, s));
    }
    if (form == FORM_SHARED) {
        EMU_TRY(launched(launch_few_tiles(in, true, false, dev.sm_count, s)));
        return launched(launch_few_tiles(out, false, true, dev.sm_count, s));
    }
    Aligned al;
    al.add(X, ldx, rows, K);
    al.add(W_in, ldwi, E * 2 * F, K);
    al.add(W_out, ldwo, E * N, F);
    const Fused f{FUSED_GATED, act, nullptr, 0, D, ldd, nullptr};
    auto products = [&] {
        Products q(rows, E);
        q.begin();
        q.add({false, E, false, rows, 0, F, K, X, ldx, W_in, ldwi, H, ldh, &f});
        q.begin();
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
    if (!fused_mode(mode) || !sizes_ok(rows, E, K, F, N)) return EMU_STATUS_NOT_SUPPORTED;
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
    if (few_bwd(rows, E, K, F, N, kPairs)) {
        // (the tiles' checks of alignment, for the same contract)
        if ((inner && !vec4_ok(dZ, lddz)) || !vec4_ok(dX, dX ? lddx : 0) || !vec4_ok(dW_in, dW_in ? lddwi : 0) ||
            !vec4_ok(dW_out, dW_out ? lddwo : 0))
            return EMU_STATUS_NOT_SUPPORTED;
        al.stand_in();  // (the copies' leading dimensions; reserve gives their addresses)
        EMU_TRY(current_device(&dev));
        EMU_TRY(al.reserve(s));
        const int M = (int)rows;
        // blocks that share a contraction or a sum, and the buffer for what they leave: the
        // contractions' in turn, the sums' until the end
        const int64_t ldf = (F + 3) & ~int64_t(3), ldk = (K + 3) & ~int64_t(3);
        const int fs = inner ? few_columns_shares(rows, E, F, N, dev.sm_count) : 1;
        const int ks = dX ? few_columns_shares(rows, E, K, 2 * F, dev.sm_count) : 1;
        const int fc = few_sums_chunk(rows, N, F, dev.sm_count), kc = few_sums_chunk(rows, 2 * F, K, dev.sm_count);
        const size_t floats_f = fs > 1 ? (size_t)fs * rows * ldf : 0, floats_k = ks > 1 ? (size_t)ks * rows * ldk : 0;
        const size_t floats_o = dW_out ? (size_t)few_sums_pieces(rows, fc) * N * ldf : 0;
        const size_t floats_i = dW_in ? (size_t)few_sums_pieces(rows, kc) * 2 * F * ldk : 0;
        const size_t floats_s = floats_f > floats_k ? floats_f : floats_k;
        float* shares = nullptr;
        if (floats_s + floats_o + floats_i) EMU_TRY(reduce_scratch(dev.id, s, floats_s + floats_o + floats_i, &shares));
        float *pieces_o = shares + floats_s, *pieces_i = pieces_o + floats_o;  // (all multiples of four floats)
        EMU_TRY(launched(al.launch(s)));
        bool after = false;
        FewSums sums[2];
        int n = 0;
        if (inner) {
            EMU_TRY(launched(launch_few_columns({M, E, offsets, F, N, dY, lddy, W_out, ldwo, D, ldd, dZ, lddz, shares, ldf}, fs,
                                                after, s)));
            after = true;
        }
        if (dW_out) {
            sums[n] = {M, E, offsets, N, F, dY, lddy, H, ldh, dW_out, lddwo, fc, pieces_o, ldf};
            EMU_TRY(launched(launch_few_sums(sums[n++], after, s)));
            after = true;
        }
        if (dX) {
            EMU_TRY(launched(launch_few_columns({M, E, offsets, K, 2 * F, dZ, lddz, W_in, ldwi, nullptr, 0, dX, lddx, shares,
                                                 ldk}, ks, after, s)));
            after = true;
        }
        if (dW_in) {
            sums[n] = {M, E, offsets, 2 * F, K, dZ, lddz, X, ldx, dW_in, lddwi, kc, pieces_i, ldk};
            EMU_TRY(launched(launch_few_sums(sums[n++], after, s)));
        }
        return launched(launch_add_pieces(sums, n, s));
    }
    Fused f{};
    auto products = [&] {
        f = {FUSED_GATED_BWD, ACT_NONE, nullptr, 0, const_cast<float*>(D), ldd, nullptr};
        Products q(rows, E);
        q.begin();
        if (inner) q.add({false, E, true, rows, 0, F, N, dY, lddy, W_out, ldwo, dZ, lddz, &f});
        if (dW_out) q.add({true, E, true, rows, N, F, 0, dY, lddy, H, ldh, dW_out, lddwo});
        if (inner) q.begin();
        if (dX) q.add({false, E, true, rows, 0, K, 2 * F, dZ, lddz, W_in, ldwi, dX, lddx});
        if (dW_in) q.add({true, E, true, rows, 2 * F, K, 0, dZ, lddz, X, ldx, dW_in, lddwi});
        return q;
    };
    return run_products(al, products, offsets, s);
}

}  // extern "C"
