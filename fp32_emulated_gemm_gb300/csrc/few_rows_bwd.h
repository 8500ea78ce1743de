// few_rows_bwd.h -- the backward products of a few rows in groups (see few_rows_bwd.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace emu {

// C[r] = A[r] B[g] for the rows r of group g (B: groups x K x N), or with D (gated, rows
// of 2N) C[r] = [A[r] B[g] | A[r] B[g]] * D[r].  Operands start on 16-byte boundaries and
// have leading dimensions that are multiples of 4.
struct FewColumns {
    int M, groups;
    const int32_t* offsets;
    int64_t N, K;
    const float* A;
    int64_t lda;
    const float* B;
    int64_t ldb;
    const float* D;  // or null
    int64_t ldd;
    float* C;
    int64_t ldc;
    float* shares = nullptr;  // shares x M rows of ldshares floats, if there are several
    int64_t ldshares = 0;
};
// C[g] = sum over the rows r of group g of A[r]^T B[r] (groups x R x N; zero for a group
// without rows); alignment likewise.  A group's rows behind its first `chunk` are summed
// by further blocks, a chunk each, in `pieces` (R x ldpieces floats for each of
// few_sums_pieces()), which launch_add_pieces adds, for up to two sums.
struct FewSums {
    int M, groups;
    const int32_t* offsets;
    int64_t R, N;
    const float* A;
    int64_t lda;
    const float* B;
    int64_t ldb;
    float* C;
    int64_t ldc;
    int chunk;
    float* pieces = nullptr;
    int64_t ldpieces = 0;
};
int few_sums_chunk(int64_t M, int64_t R, int64_t N, int sm_count);
inline int64_t few_sums_pieces(int64_t M, int chunk) { return (M - 1) / chunk; }
// `after_own`: the launch follows one of these, with nothing in between.
// `shares`: blocks that share a contraction, few_columns_shares() or less.
int few_columns_shares(int64_t M, int64_t groups, int64_t N, int64_t K, int sm_count);
cudaError_t launch_few_columns(const FewColumns& p, int shares, bool after_own, cudaStream_t stream);
cudaError_t launch_few_sums(const FewSums& p, bool after_own, cudaStream_t stream);
// (Behind the sums' launches or others of these; nothing if there can be no pieces.)
cudaError_t launch_add_pieces(const FewSums* sums, int n, cudaStream_t stream);

}  // namespace emu
