// gemm_epi.h -- the emulated-GEMM kernels with a fused epilogue (EPI_ACT,
// EPI_GATED, EPI_GATED_BWD of emu_kernel.cuh).  Each epilogue's kernels are
// compiled in a source file of their own, which hands them to the host side
// as a table.
#pragma once

#include <cuda_runtime.h>

#include "emu_kernel.cuh"

namespace emu {

struct EpiTable {
    cudaError_t (*set_attributes)();  // once per device, before the first launch
    // mode BF16X9 or TF32X3, any pipeline shape of make_plan
    cudaError_t (*launch)(int mode, int pipe, cudaLaunchConfig_t cfg, const Params& p);
};
extern const EpiTable kEpiAct, kEpiGated, kEpiGatedBwd;
// Grouped products (GROUP_ROWS with each epilogue of the experts, GROUP_SUM):
// BF16x9 and unpacked shapes alone.
extern const EpiTable kRowsStore, kRowsGated, kRowsGatedBwd, kSumStore;

// The TF32 modes have one unpacked and one packed shape (PIPE_LONG_K* read as
// PIPE_SHORT_K*); BF16x9 is never split ahead of a product.
template <int MODE, int PIPE, int EPI>
cudaError_t epi_set_attribute() {
    return cudaFuncSetAttribute(emu_gemm_kernel<MODE, PIPE, false, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem_bytes<MODE, PIPE>());
}
template <int EPI> cudaError_t epi_set_attributes() {
    cudaError_t e = epi_set_attribute<MODE_BF16X9, PIPE_SHORT_K, EPI>();
    if (e == cudaSuccess) e = epi_set_attribute<MODE_BF16X9, PIPE_LONG_K, EPI>();
    if (e == cudaSuccess) e = epi_set_attribute<MODE_TF32X3, PIPE_SHORT_K, EPI>();
    if (e == cudaSuccess) e = epi_set_attribute<MODE_TF32X3, PIPE_SHORT_K_PACKED, EPI>();
    return e;
}
template <int MODE, int PIPE, int EPI>
cudaError_t epi_launch_one(cudaLaunchConfig_t cfg, const Params& p) {
    cfg.dynamicSmemBytes = smem_bytes<MODE, PIPE>();
    return cudaLaunchKernelEx(&cfg, emu_gemm_kernel<MODE, PIPE, false, EPI>, p);
}
template <int EPI> cudaError_t epi_launch(int mode, int pipe, cudaLaunchConfig_t cfg, const Params& p) {
    if (mode == MODE_TF32X3)
        return pipe_packed(pipe) ? epi_launch_one<MODE_TF32X3, PIPE_SHORT_K_PACKED, EPI>(cfg, p)
                                 : epi_launch_one<MODE_TF32X3, PIPE_SHORT_K, EPI>(cfg, p);
    return pipe == PIPE_LONG_K ? epi_launch_one<MODE_BF16X9, PIPE_LONG_K, EPI>(cfg, p)
                               : epi_launch_one<MODE_BF16X9, PIPE_SHORT_K, EPI>(cfg, p);
}

template <int MODE, int PIPE, int EPI, int GROUP>
cudaError_t group_set_attribute() {
    return cudaFuncSetAttribute(emu_gemm_kernel<MODE, PIPE, false, EPI, GROUP>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<MODE, PIPE>());
}
template <int EPI, int GROUP> cudaError_t group_set_attributes() {
    cudaError_t e = group_set_attribute<MODE_BF16X9, PIPE_SHORT_K, EPI, GROUP>();
    if (e == cudaSuccess) e = group_set_attribute<MODE_BF16X9, PIPE_LONG_K, EPI, GROUP>();
    return e;
}
template <int MODE, int PIPE, int EPI, int GROUP>
cudaError_t group_launch_one(cudaLaunchConfig_t cfg, const Params& p) {
    cfg.dynamicSmemBytes = smem_bytes<MODE, PIPE>();
    return cudaLaunchKernelEx(&cfg, emu_gemm_kernel<MODE, PIPE, false, EPI, GROUP>, p);
}
template <int EPI, int GROUP> cudaError_t group_launch(int, int pipe, cudaLaunchConfig_t cfg, const Params& p) {
    return pipe == PIPE_LONG_K ? group_launch_one<MODE_BF16X9, PIPE_LONG_K, EPI, GROUP>(cfg, p)
                               : group_launch_one<MODE_BF16X9, PIPE_SHORT_K, EPI, GROUP>(cfg, p);
}

}  // namespace emu
