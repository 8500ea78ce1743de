// internal.h -- what the library's source files share on the host side.  Not
// part of the C ABI (include/emu_gemm.h).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/emu_gemm.h"

namespace emu {

// The current device, bound to this host thread and checked to be sm_103.
struct DeviceCtx { int id, sm_count; };
emu_status_t current_device(DeviceCtx* out);

// The (device, stream)'s buffer for column-sum partials, at least `floats`
// long: grown on demand, kept until emu_shutdown().  Not the split-K
// workspace, which a product on the same stream may be using in between.
emu_status_t reduce_scratch(int dev, cudaStream_t stream, size_t floats, float** out);

// One product C = op(A) op(B) + beta C + bias as the public entry points run
// it.  `check` true: argument checks and buffer reservation alone, so that an
// operator of several launches can make sure of all of them before the first.
struct Gemm {
    bool a_mn, b_mn;
    int64_t M, N, K;
    const float *A;
    int64_t lda;
    const float *B;
    int64_t ldb;
    float beta;
    float *C;
    int64_t ldc;
    const float *bias;
};
emu_status_t gemm(emu_mode_t mode, const Gemm& g, cudaStream_t stream, bool check);

}  // namespace emu
