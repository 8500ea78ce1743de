// gemm_rows_gated_bwd.cu -- the emulated-GEMM kernels with rows in groups and the EPI_GATED_BWD epilogue.
#include "gemm_epi.h"

namespace emu {
const EpiTable kRowsGatedBwd = {group_set_attributes<EPI_GATED_BWD, GROUP_ROWS>, group_launch<EPI_GATED_BWD, GROUP_ROWS>};
}
