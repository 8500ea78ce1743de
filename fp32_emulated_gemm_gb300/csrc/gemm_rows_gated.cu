// gemm_rows_gated.cu -- the emulated-GEMM kernels with rows in groups and the EPI_GATED epilogue.
#include "gemm_epi.h"

namespace emu {
const EpiTable kRowsGated = {group_set_attributes<EPI_GATED, GROUP_ROWS>, group_launch<EPI_GATED, GROUP_ROWS>};
}
