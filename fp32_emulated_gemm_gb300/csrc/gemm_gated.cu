// gemm_gated.cu -- the emulated-GEMM kernels with the EPI_GATED epilogue.
#include "gemm_epi.h"

namespace emu {
const EpiTable kEpiGated = {epi_set_attributes<EPI_GATED>, epi_launch<EPI_GATED>};
}
