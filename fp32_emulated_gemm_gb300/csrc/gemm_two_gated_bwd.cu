// gemm_two_gated_bwd.cu -- the emulated-GEMM kernels with rows in groups and the EPI_GATED_BWD epilogue
// beside a sum over the groups' rows.
#include "gemm_epi.h"

namespace emu {
const TwoTable kTwoGatedBwd = {two_set_attributes<EPI_GATED_BWD>, two_launch<EPI_GATED_BWD>};
}
