// gemm_rows.cu -- the emulated-GEMM kernels with rows in groups and the plain epilogue.
#include "gemm_epi.h"

namespace emu {
const EpiTable kRowsStore = {group_set_attributes<EPI_STORE, GROUP_ROWS>, group_launch<EPI_STORE, GROUP_ROWS>};
}
