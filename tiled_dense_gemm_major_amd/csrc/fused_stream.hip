// libtgemm: the streaming kernels over rows of groups.
#include "fused_launch.hpp"
#include "fused_stream.hpp"

namespace tgemm_fused {

hipError_t rows_stream(int dtype, int layout, Form form, const FusedArgs& p, int64_t tiles_m, int tiles_n, hipStream_t s) {
    const dim3 grid((unsigned)(tiles_m * tiles_n));
#define STREAM(DT, MT, NT, NW, S, OCC)                                                     \
    hipLaunchKernelGGL((tgemm::fused_stream<DT, MT, NT, NW, S, OCC>), grid, dim3(NW * 64), 0, s, p, tiles_n)
#define FORM(MT, NT, NW, S, OCC)                                                           \
    do {                                                                                   \
        if (dtype == tgemm::DT_F16)                                                        \
            STREAM(0, MT, NT, NW, S, OCC);                                                 \
        else                                                                               \
            STREAM(1, MT, NT, NW, S, OCC);                                                 \
    } while (0)
    if (layout == tgemm::LAYOUT_KN) {
#define STREAM_KN(DT, MT, NW, S, OCC)                                                      \
    hipLaunchKernelGGL((tgemm::fused_stream_kn<DT, MT, NW, S, OCC>), grid, dim3(NW * 64), 0, s, p, tiles_n)
        if (form == FORM_STREAM32) {
            if (dtype == tgemm::DT_F16)
                STREAM_KN(0, 1, 4, 2, 2);
            else
                STREAM_KN(1, 1, 4, 2, 2);
        } else {
            if (dtype == tgemm::DT_F16)
                STREAM_KN(0, 2, 4, 3, 1);
            else
                STREAM_KN(1, 2, 4, 3, 1);
        }
#undef STREAM_KN
        return hipGetLastError();
    }
    switch (form) {
    case FORM_STREAM16: FORM(1, 2, 4, 3, 2); break;
    case FORM_STREAM16_2: FORM(1, 2, 2, 3, 2); break;
    case FORM_STREAM32: FORM(2, 2, 4, 2, 2); break;
    default: FORM(4, 2, 4, 3, 1); break;
    }
#undef FORM
#undef STREAM
    return hipGetLastError();
}

}  // namespace tgemm_fused
