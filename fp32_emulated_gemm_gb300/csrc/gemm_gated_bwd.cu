// gemm_gated_bwd.cu -- the emulated-GEMM kernels with the EPI_GATED_BWD epilogue.
#include "gemm_epi.h"

namespace emu {
const EpiTable kEpiGatedBwd = {epi_set_attributes<EPI_GATED_BWD>, epi_launch<EPI_GATED_BWD>};
}
