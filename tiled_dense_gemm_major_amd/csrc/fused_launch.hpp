// libtgemm: the compiled forms of the fused and grouped kernels, by translation unit.
#pragma once

#include "fused.hpp"

namespace tgemm_fused {

using tgemm::FusedArgs;
using tgemm::SlopeArgs;
using tgemm::SumArgs;

// Tile forms of the tiled kernels.
enum Form {
    FORM_QUAD = 0,       // 256 x 256, one wave per SIMD
    FORM_QUAD192 = 1,    // 192 x 256
    FORM_128 = 2,        // 128 x 128, four waves, two stages: two workgroups per compute unit
    FORM_128_DEEP = 3,   // the same in four stages, alone on its compute unit
    FORM_64 = 4,         // 64 x 128, four waves, three stages
    FORM_SMALL = 5,      // 64 x 64, two waves, three stages
    FORM_SMALL_DEEP = 6, // the same in eight
    FORM_STREAM16 = 7,   // B [N,K]: 16 rows, 32 columns, K split over four waves
    FORM_STREAM16_2 = 8, // the same over two waves
    FORM_STREAM32 = 9,   // 32 rows, 32 columns, four waves (either B)
    FORM_STREAM64 = 10,  // 64 rows, 32 columns, four waves (either B)
    FORMS = 11
};
struct Tile {
    int m, n;
};
constexpr Tile kTiles[FORMS] = {{256, 256}, {192, 256}, {128, 128}, {128, 128}, {64, 128}, {64, 64},
                                {64, 64},   {16, 32},   {16, 32},   {32, 32},  {64, 32}};
constexpr bool form_takes(Form f, int layout) { return layout == 0 || (f != FORM_STREAM16 && f != FORM_STREAM16_2); }

// Forms of the sums over a group's rows.
enum SumForm {
    SUM_QUAD = 0,        // 256 x 256, the quad kernel (no row index)
    SUM_256 = 1,         // 256 x 256, eight waves
    SUM_128 = 2,         // 128 x 128, four waves, two stages
    SUM_SMALL = 3,       // 64 x 64, two waves, four stages
    SUM_FORMS = 4
};
constexpr int kSumTiles[SUM_FORMS] = {256, 256, 128, 64};

// One launch of a tiled kernel over rows of groups with B [N,K] or [K,N]; `tiles_m` is an
// upper bound on the row tiles of all groups.
hipError_t rows_tiled_nk(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);
hipError_t rows_quad_nk(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);
hipError_t rows_quad_kn(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);
hipError_t rows_stream(int dtype, int layout, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);
hipError_t rows_tiled_kn(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s);

// One launch of a sum over a group's rows (not SUM_QUAD, which is sum_quad).
hipError_t sum_tiled(int dtype, SumForm form, const SumArgs& p, hipStream_t s);

hipError_t sum_quad(int dtype, const SumArgs& p, hipStream_t s);

}  // namespace tgemm_fused
