// libtgemm: the compiled forms of the fused and grouped kernels, by translation unit.
#pragma once

#include "fused.hpp"

namespace tgemm_fused {

using tgemm::FusedArgs;
using tgemm::SlopeArgs;
using tgemm::SumArgs;

// Tile forms of the tiled kernels.
enum Form { FORM_256 = 0, FORM_128 = 1, FORM_64 = 2, FORMS = 3 };
struct Tile {
    int m, n;
};
constexpr Tile kTiles[FORMS] = {{256, 256}, {128, 128}, {64, 128}};

// One launch of a tiled kernel over rows of groups with B [N,K] or [K,N]; `tiles_m` is an
// upper bound on the row tiles of all groups.
hipError_t rows_tiled_nk(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);
hipError_t rows_tiled_kn(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);

// One launch of the tiled sum over a group's rows (FORM_256 or FORM_128).
hipError_t sum_tiled(int dtype, Form form, const SumArgs& p, hipStream_t s);

}  // namespace tgemm_fused
