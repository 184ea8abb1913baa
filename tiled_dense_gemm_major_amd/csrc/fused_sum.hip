// libtgemm: the tiled kernels that sum over a group's rows.
#include "fused_launch.hpp"
#include "fused_tile.hpp"

namespace tgemm_fused {

hipError_t sum_tiled(int dtype, SumForm form, const SumArgs& p, hipStream_t s) {
#define SUM(DT, BI, BJ, WI, WJ, ST, OCC)                                                   \
    do {                                                                                   \
        const int gi = (p.I + BI - 1) / BI, gj = (p.J + BJ - 1) / BJ;                      \
        hipLaunchKernelGGL((tgemm::sum_tiled<DT, BI, BJ, WI, WJ, ST, OCC>),                \
                           dim3((unsigned)((int64_t)p.groups * p.parts * gi * gj)), dim3(WI * WJ * 64), 0, s, p, gi, gj); \
    } while (0)
#define FORM(BI, BJ, WI, WJ, ST, OCC)                                                      \
    do {                                                                                   \
        if (dtype == tgemm::DT_F16)                                                        \
            SUM(0, BI, BJ, WI, WJ, ST, OCC);                                               \
        else                                                                               \
            SUM(1, BI, BJ, WI, WJ, ST, OCC);                                               \
    } while (0)
    switch (form) {
    case SUM_128: FORM(128, 128, 2, 2, 2, 2); break;
    case SUM_SMALL: FORM(64, 64, 2, 1, 4, 2); break;
    default: FORM(256, 256, 2, 4, 2, 2); break;
    }
#undef FORM
#undef SUM
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.parts == 1)
        return e;
    const dim3 grid((unsigned)(((int64_t)p.groups * p.I * (p.J / 8) + 255) / 256));
    if (dtype == tgemm::DT_F16)
        hipLaunchKernelGGL((tgemm::sum_parts<0>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((tgemm::sum_parts<1>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace tgemm_fused
