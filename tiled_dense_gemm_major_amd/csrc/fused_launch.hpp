// libtgemm: the compiled forms of the fused and grouped kernels, by translation unit.
#pragma once

#include "fused.hpp"

namespace tgemm_fused {

using tgemm::FusedArgs;
using tgemm::SlopeArgs;
using tgemm::SumArgs;

// Tile forms of the tiled kernels.
enum Form {
    FORM_QUAD = 0,      // 256 x 256, one wave per SIMD
    FORM_128 = 1,       // 128 x 128, four waves
    FORM_64 = 2,        // 64 x 128, four waves
    FORM_SMALL = 3,     // 64 x 64, two waves
    FORM_STREAM16 = 4,  // 16 rows, 32 columns, K split over four waves (B [N,K] only)
    FORM_STREAM16_2 = 5,// the same over two waves
    FORM_STREAM32 = 6,  // 32 rows, 32 columns, four waves
    FORM_STREAM64 = 7,  // 64 rows, 32 columns, four waves
    FORMS = 8
};
struct Tile {
    int m, n;
};
constexpr Tile kTiles[FORMS] = {{256, 256}, {128, 128}, {64, 128}, {64, 64}, {16, 32}, {16, 32}, {32, 32}, {64, 32}};

// One launch of a tiled kernel over rows of groups with B [N,K] or [K,N]; `tiles_m` is an
// upper bound on the row tiles of all groups.
hipError_t rows_tiled_nk(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);
hipError_t rows_quad(int dtype, int layout, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);
hipError_t rows_stream(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);
hipError_t rows_tiled_kn(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);

// One launch of the tiled sum over a group's rows (256 x 256 or 128 x 128 tiles).
hipError_t sum_tiled(int dtype, bool large, const SumArgs& p, hipStream_t s);

hipError_t sum_quad(int dtype, const SumArgs& p, hipStream_t s);

}  // namespace tgemm_fused
