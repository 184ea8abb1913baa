// libtgemm: the launchers of the fused and grouped kernels, one per compiled form.
#pragma once

#include "fused.hpp"

namespace tgemm_fused {

using tgemm::FusedArgs;
using tgemm::SlopeArgs;
using tgemm::SumArgs;

// The launch of one form over rows of groups (`grid` workgroups, an upper bound on the
// tiles) or of one summing over them.
typedef hipError_t (*rows_fn)(const FusedArgs& p, int64_t grid, int grid_n, hipStream_t s);
typedef hipError_t (*sum_fn)(const SumArgs& p, hipStream_t s);

}  // namespace tgemm_fused
