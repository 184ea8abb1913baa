// libtgemm: the quad kernel summing over a group's rows.
#include "fused_launch.hpp"
#include "fused_tile.hpp"

namespace tgemm_fused {

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
