// libtgemm: the tiled kernels over rows of groups, B [N,K].
#include "fused_launch.hpp"
#include "fused_tile.hpp"

namespace tgemm_fused {

hipError_t rows_tiled_nk(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s) {
    const dim3 grid((unsigned)(tiles_m * tiles_n));
#define TILED(DT, BM, BN, WM, WN, ST, OCC, G)                                              \
    hipLaunchKernelGGL((tgemm::fused_tiled<DT, tgemm::LAYOUT_NK, BM, BN, WM, WN, ST, OCC>), grid, \
                       dim3(WM * WN * 64), 0, s, p, tiles_n, G)
#define FORM(BM, BN, WM, WN, ST, OCC, G)                                                   \
    do {                                                                                   \
        if (dtype == tgemm::DT_F16)                                                        \
            TILED(0, BM, BN, WM, WN, ST, OCC, G);                                          \
        else                                                                               \
            TILED(1, BM, BN, WM, WN, ST, OCC, G);                                          \
    } while (0)
    switch (form) {
    case FORM_128: FORM(128, 128, 2, 2, 2, 2, 8); break;
    case FORM_128_DEEP: FORM(128, 128, 2, 2, 4, 1, 8); break;
    case FORM_64: FORM(64, 128, 2, 2, 3, 2, 8); break;
    case FORM_SMALL: FORM(64, 64, 2, 1, 3, 2, 8); break;
    default: FORM(64, 64, 2, 1, 8, 1, 8); break;
    }
#undef FORM
#undef TILED
    return hipGetLastError();
}

}  // namespace tgemm_fused
