// internal.h -- what the library's source files share on the host side.  Not
// part of the C ABI (include/emu_gemm.h).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "../../include/emu_gemm.h"

namespace emu {

// The current device, bound to this host thread and checked to be sm_103.
struct DeviceCtx { int id, sm_count; };
emu_status_t current_device(DeviceCtx* out);

// Whether launches may overlap the end of the kernel before them on the stream
// (programmatic dependent launch; EMU_PDL=0 turns it off).
bool pdl_enabled();

// Held by an entry point from its first use of a stream's library buffers (or
// its side stream and events) to its last launch: calls of several host threads
// on one stream share those, and their launches must not come between one
// another.  Not recursive.  Calls on different streams seldom share a lock.
class StreamLock {
public:
    explicit StreamLock(cudaStream_t stream);

private:
    std::lock_guard<std::mutex> lock_;
};

// The (device, stream)'s buffer for column-sum partials, at least `floats`
// long: grown on demand (never under capture), kept until emu_shutdown().  Not
// the split-K workspace, which a product on the same stream may be using in
// between.
emu_status_t reduce_scratch(int dev, cudaStream_t stream, size_t floats, float** out);

// Likewise its buffer for aligned copies of operands.
emu_status_t align_scratch(int dev, cudaStream_t stream, size_t floats, float** out);

// What a product's epilogue does besides the bias (the Epi kinds of
// emu_kernel.cuh; modes BF16x9 and TF32x3, K > 0).
struct Fused {
    int kind;           // a FusedKind
    int act;
    const float *res;   // FUSED_ACT: R, or null
    int64_t ldr;
    float *d;           // the derivative's factors D: written when not null (FUSED_GATED_BWD: read)
    int64_t ldd;
    float *sums;        // FUSED_GATED_BWD: ceil(M / 32) x 2N partial column sums, or null
};
enum FusedKind : int { FUSED_ACT = 1, FUSED_GATED = 2, FUSED_GATED_BWD = 3 };
inline bool fused_mode(emu_mode_t mode) { return mode == EMU_MODE_BF16X9 || mode == EMU_MODE_TF32X3; }

// How far a product's call goes, so that an operator of several launches can make
// sure of all of them before the first: its arguments' checks (nothing that needs
// the device), the reservation of its buffers, its launches.
enum Until { UNTIL_CHECKED, UNTIL_RESERVED, UNTIL_LAUNCHED };

// One product C = op(A) op(B) + beta C + bias as the public entry points run it.
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
    const Fused *fused = nullptr;  // FUSED_GATED: N is F, B has 2F rows and the bias 2F values
};
emu_status_t gemm(emu_mode_t mode, const Gemm& g, cudaStream_t stream, Until until);

// Two independent products, each `after` work queued on `stream` before the call
// and both before work queued after it: side by side on shares of the GPU when
// that is predicted faster than one after the other.  Either may be absent (null).
emu_status_t gemm_two(emu_mode_t mode, const Gemm* a, const Gemm* b, cudaStream_t stream, Until until);

}  // namespace emu
