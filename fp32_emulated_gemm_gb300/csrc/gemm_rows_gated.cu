// gemm_rows_gated.cu -- the emulated-GEMM kernels with rows in groups and the EPI_GATED epilogue.
#include "gemm_epi.h"

namespace emu {
const EpiTable kRowsGated = {rows_set_attributes<EPI_GATED>, rows_launch<EPI_GATED>};
}
