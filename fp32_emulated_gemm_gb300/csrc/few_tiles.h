// few_tiles.h -- the forward products of some rows in groups (see few_tiles.cu).
#pragma once

#include "few_rows.h"

namespace emu {

// As launch_few_rows_grouped; rows of X and W on 16-byte boundaries, K a multiple of 4.
bool few_tiles_fit(const FewRows& p);
cudaError_t launch_few_tiles(const FewRows& p, bool gated, bool after_own, int sm_count, cudaStream_t stream);

}  // namespace emu
