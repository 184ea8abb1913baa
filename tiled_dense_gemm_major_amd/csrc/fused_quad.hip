// libtgemm: the quad kernel over rows of groups and summing over them.
#include "fused_launch.hpp"
#include "fused_tile.hpp"

namespace tgemm_fused {

hipError_t rows_quad(int dtype, int layout, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s) {
    const dim3 grid((unsigned)(tiles_m * tiles_n));
    // the instruction-offset form of the loads: rows of 64 elements or more (B [K,N]: 256),
    // and A rows in order
    const bool offs = !p.row_index && p.lda >= 64 && p.ldb >= (layout == 0 ? 64 : 256);
#define QUAD(DT, MF, L, OFFS)                                                              \
    hipLaunchKernelGGL((tgemm::fused_quad<DT, MF, L, OFFS>), grid, dim3(256), 0, s, p, tiles_n, 4)
#define QUAD_L(DT, OFFS)                                                                   \
    if (layout == 0)                                                                       \
        QUAD(DT, 16, 0, OFFS);                                                             \
    else                                                                                   \
        QUAD(DT, 32, 1, OFFS);
    if (dtype == tgemm::DT_F16) {
        if (offs) {
            QUAD_L(0, true)
        } else {
            QUAD_L(0, false)
        }
    } else {
        if (offs) {
            QUAD_L(1, true)
        } else {
            QUAD_L(1, false)
        }
    }
#undef QUAD_L
#undef QUAD
    return hipGetLastError();
}

hipError_t sum_quad(int dtype, const SumArgs& p, hipStream_t s) {
    const int gi = (p.I + 255) / 256, gj = (p.J + 255) / 256;
    const dim3 grid((unsigned)((int64_t)p.groups * gi * gj));
    const bool offs = p.ldl >= 256 && p.ldr >= 256;
#define QUAD(DT, OFFS) hipLaunchKernelGGL((tgemm::sum_quad<DT, OFFS>), grid, dim3(256), 0, s, p, gi, gj)
    if (dtype == tgemm::DT_F16) {
        if (offs)
            QUAD(0, true);
        else
            QUAD(0, false);
    } else {
        if (offs)
            QUAD(1, true);
        else
            QUAD(1, false);
    }
#undef QUAD
    return hipGetLastError();
}

}  // namespace tgemm_fused
