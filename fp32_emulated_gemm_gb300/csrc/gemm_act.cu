// gemm_act.cu -- the emulated-GEMM kernels with the EPI_ACT epilogue.
#include "gemm_epi.h"

namespace emu {
const EpiTable kEpiAct = {epi_set_attributes<EPI_ACT>, epi_launch<EPI_ACT>};
}
