// aligned.cuh -- copies of operands whose rows TMA cannot address.
#pragma once

#include <cuda_runtime.h>

#include "internal.h"
#include "row_ops.cuh"

namespace emu {
namespace {

constexpr int kCopyWarps = 8;

// Copies of matrices, a warp a row at a time.
struct CopyJob {
    const float* src;
    int64_t lds;
    float* dst;
    int64_t ldd, rows, cols;
};
constexpr int kMaxCopies = 7;
struct CopyJobs { int n; CopyJob job[kMaxCopies]; };
__global__ void __launch_bounds__(32 * kCopyWarps) copy_rows_kernel(const __grid_constant__ CopyJobs jobs) {
    int64_t r = blockIdx.x * (int64_t)kCopyWarps + threadIdx.y;
    for (int i = 0; i < jobs.n; ++i) {
        const CopyJob& j = jobs.job[i];
        for (; r < j.rows; r += (int64_t)gridDim.x * kCopyWarps) {
            const float* src = j.src + r * j.lds;
            float* dst = j.dst + r * j.ldd;
            for (int64_t c = threadIdx.x; c < j.cols; c += 32 * 8) {  // eight words of a lane in flight
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + 32 * k < j.cols) v[k] = __ldg(src + c + 32 * k);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + 32 * k < j.cols) dst[c + 32 * k] = v[k];
            }
        }
        r -= j.rows;
    }
}

// Operands of the products (TMA) whose rows do not start on 16-byte boundaries
// are read from copies that do, in a buffer of the library's, reserved once the
// call's other arguments have been checked: all of a call's by one launch ahead of its first product (block forward, three copies, 3740 x
// 169, F = 320, TF32x3: 53 us; with a copy each by the caller 103 us).
class Aligned {
public:
    void add(const float*& p, int64_t& ld, int64_t rows, int64_t cols) {
        if (!p || rows < 1 || cols < 1 || ld < cols || vec4_ok(p, rows > 1 ? ld : 0)) {
            if (rows == 1 && p && ld >= cols) ld = (ld + 3) & ~int64_t(3);  // one row: any stride
            return;
        }
        CopyJob& j = jobs_.job[jobs_.n];
        j = {p, ld, nullptr, (cols + 3) & ~int64_t(3), rows, cols};
        p_[jobs_.n] = &p;
        ld_[jobs_.n++] = &ld;
        floats_ += (size_t)rows * j.ldd;
    }
    void add_vector(const float*& p, int64_t n) {
        int64_t& ld = vector_ld_[vectors_++];
        ld = n;
        add(p, ld, 1, n);
    }
    // The operands' addresses for the checks of a call's arguments: any that a
    // copy could have.
    void stand_in() {
        for (int i = 0; i < jobs_.n; ++i) {
            *p_[i] = reinterpret_cast<const float*>(uintptr_t(256));
            *ld_[i] = jobs_.job[i].ldd;
        }
    }
    // After the checks: the copies' addresses take the place of the operands'.
    emu_status_t reserve(cudaStream_t s) {
        if (jobs_.n == 0) return EMU_STATUS_SUCCESS;
        DeviceCtx dev;
        emu_status_t st = current_device(&dev);
        float* base = nullptr;
        if (st == EMU_STATUS_SUCCESS) st = align_scratch(dev.id, s, floats_, &base);
        if (st != EMU_STATUS_SUCCESS) return st;
        for (int i = 0; i < jobs_.n; ++i) {
            CopyJob& j = jobs_.job[i];
            j.dst = base;
            *p_[i] = base;
            base += j.rows * j.ldd;
            rows_ += j.rows;
        }
        const int64_t blocks = (rows_ + kCopyWarps - 1) / kCopyWarps;
        blocks_ = (unsigned)(blocks < dev.sm_count * 8 ? blocks : dev.sm_count * 8);
        return EMU_STATUS_SUCCESS;
    }
    cudaError_t launch(cudaStream_t s) const {
        if (jobs_.n == 0) return cudaSuccess;
        cudaGetLastError();
        copy_rows_kernel<<<blocks_, dim3(32, kCopyWarps), 0, s>>>(jobs_);
        return cudaGetLastError();
    }

private:
    CopyJobs jobs_{};
    const float** p_[kMaxCopies];
    int64_t* ld_[kMaxCopies];
    int64_t vector_ld_[2], rows_ = 0;
    int vectors_ = 0;
    size_t floats_ = 0;
    unsigned blocks_ = 0;
};

}  // namespace
}  // namespace emu
