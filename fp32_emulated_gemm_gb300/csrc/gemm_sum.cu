// gemm_sum.cu -- the emulated-GEMM kernels with the contraction in groups.
#include "gemm_epi.h"

namespace emu {
const EpiTable kSumStore = {group_set_attributes<EPI_STORE, GROUP_SUM>, group_launch<EPI_STORE, GROUP_SUM>};
}
