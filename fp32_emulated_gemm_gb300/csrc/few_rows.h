// few_rows.h -- the forward pass of a layer for a few tokens (see few_rows.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "activation.cuh"

namespace emu {

// A forward pass of few enough multiplications runs on the CUDA cores instead of
// in 256-row tiles: N counts every column of the weight (both halves of a gated
// one).  The tiles take 14 us or more, this form 3 us and 0.2 us for each
// million multiplications, measured for 1 to 64 rows of layers from 256 x 1024
// to 2048 x 8192 (see few_rows.cu); the bound on M keeps to that range of
// shapes.
constexpr double kFewRowsFma = 50e6;
constexpr int64_t kFewRowsMax = 1024;
bool few_rows_fit(int64_t M, int64_t N, int64_t K);

// Y = a(X W^T + bias) + R, or with `gated` (N = F, W of 2F rows, bias of 2F
// values) Y = a(G) U; D as in emu_linear_act_fwd and emu_gated_fwd.  Any
// alignment; M, N > 0 within few_rows_fit.  `after_own`: the launch follows this library's
// kernel that writes X, itself launched without overlap, and nothing in
// between: it may read W while that one finishes.
struct FewRows {
    int M;
    int64_t N, K;
    const float* X;
    int64_t ldx;
    const float* W;
    int64_t ldw;
    const float* bias;
    const float* R;
    int64_t ldr;
    float* D;
    int64_t ldd;
    float* Y;
    int64_t ldy;
    ActParams act;
};
cudaError_t launch_few_rows(const FewRows& p, bool gated, bool after_own, int sm_count, cudaStream_t stream);

}  // namespace emu
