// The kernels of products with 4-bit integer weights.
#include "int4.hpp"

namespace sg {

constexpr int kInt4Waves = 8;

template <int DT, int GROUP>
static hipError_t launch_group(int mt, int nt, const Int4Params& x, unsigned blocks,
                               hipStream_t st) {
#define SG_INT4_CASE(MT, NT)                                                                  \
    if (mt == MT && nt == NT) {                                                               \
        hipLaunchKernelGGL((int4_kernel<DT, GROUP, MT, NT, kInt4Waves>), dim3(blocks),        \
                           dim3(64 * kInt4Waves), 0, st, x);                                  \
        return hipGetLastError();                                                             \
    }
    SG_INT4_CASE(1, 1)
    SG_INT4_CASE(1, 2)
    SG_INT4_CASE(1, 4)
    SG_INT4_CASE(2, 2)
    SG_INT4_CASE(2, 4)
#undef SG_INT4_CASE
    return hipErrorInvalidValue;
}

template <int DT>
static hipError_t launch_dt(int group, int mt, int nt, const Int4Params& x, unsigned blocks,
                            hipStream_t st) {
    if (group == 32) return launch_group<DT, 32>(mt, nt, x, blocks, st);
    if (group == 64) return launch_group<DT, 64>(mt, nt, x, blocks, st);
    return launch_group<DT, 128>(mt, nt, x, blocks, st);
}

hipError_t launch_int4(int dt, int group, int mt, int nt, const Int4Params& x, unsigned blocks,
                       hipStream_t st) {
    return dt == DT_F16 ? launch_dt<DT_F16>(group, mt, nt, x, blocks, st)
                        : launch_dt<DT_BF16>(group, mt, nt, x, blocks, st);
}

}  // namespace sg
