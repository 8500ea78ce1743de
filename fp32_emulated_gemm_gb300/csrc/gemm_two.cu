// gemm_two.cu -- the emulated-GEMM kernels with rows in groups beside a sum over the groups' rows.
#include "gemm_epi.h"

namespace emu {
const TwoTable kTwoStore = {two_set_attributes<EPI_STORE>, two_launch<EPI_STORE>};
}
