// gemm_rows.cu -- the emulated-GEMM kernels with rows in groups and the plain epilogue.
#include "gemm_epi.h"

namespace emu {
const EpiTable kRowsStore = {rows_set_attributes<EPI_STORE>, rows_launch<EPI_STORE>};
}
