// few_rows.h -- the forward pass of a layer for a few tokens (see few_rows.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "activation.cuh"

namespace emu {

// A forward pass of few enough rows runs on the CUDA cores instead of in 256-row
// tiles; N counts every column of the weight (both halves of a gated one).
// Measured from 1 to 64 rows and from 256 x 1024 to 1024 x 40000 weights, this
// form takes 3 us and, for a million weights, 0.65 us at one row to 1.5 us at
// eight and 0.19 us a row from there; the tiles take 14 us and 2.2 us for a
// million weights.  So up to eight rows always, and more while (M - 8) N K is
// within the 11 us between the fixed costs; the bound on M keeps to shapes
// like the measured ones.
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
