// libtgemm: the quad kernel over rows of groups, B [K,N].
#include "fused_launch.hpp"
#include "fused_tile.hpp"

namespace tgemm_fused {

hipError_t rows_quad_kn(int dtype, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s) {
    const dim3 grid((unsigned)(tiles_m * tiles_n));
    // the instruction-offset form of the loads: rows of 64 elements or more (B [K,N]: 256),
    // and A rows in order
    const bool offs = !p.row_index && p.lda >= 64 && p.ldb >= 256;
#define QUAD(DT, OFFS, BMT)                                                                \
    hipLaunchKernelGGL((tgemm::fused_quad<DT, 32, 1, OFFS, BMT>), grid, dim3(256), 0, s, p, tiles_n, 4)
#define QUAD_ROWS(DT, OFFS)                                                                \
    if (form == FORM_QUAD)                                                                 \
        QUAD(DT, OFFS, 256);                                                               \
    else                                                                                   \
        QUAD(DT, OFFS, 192);
    if (dtype == tgemm::DT_F16) {
        if (offs) {
            QUAD_ROWS(0, true)
        } else {
            QUAD_ROWS(0, false)
        }
    } else {
        if (offs) {
            QUAD_ROWS(1, true)
        } else {
            QUAD_ROWS(1, false)
        }
    }
#undef QUAD_ROWS
#undef QUAD
    return hipGetLastError();
}

}  // namespace tgemm_fused
