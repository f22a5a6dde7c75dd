// launch_int4.hpp -- host launcher of the kernels of products with 4-bit integer weights, one
// translation unit for each operand type with and without zero points.
#pragma once

#include "int4.hpp"

namespace sg {

template <int DT, bool ZEROS, int GROUP>
hipError_t launch_int4_group(int cfg, const Int4Params& x, unsigned blocks, hipStream_t st) {
#define SG_INT4_CASE(ID, MT, NT, NW, ...)                                           \
    case ID:                                                                        \
        hipLaunchKernelGGL((int4_kernel<DT, GROUP, ZEROS, MT, NT, NW>),             \
                           dim3(blocks), dim3(64 * NW), 0, st, x);                  \
        return hipGetLastError();
#define SG_INT4_TILE(ID, MT, NT, NW, ...)                                           \
    case ID:                                                                        \
        hipLaunchKernelGGL((int4_tile_kernel<DT, GROUP, ZEROS, MT / 2, NW / 4>),    \
                           dim3(blocks), dim3(64 * NW), 0, st, x);                  \
        return hipGetLastError();
    switch (cfg) {
        SG_INT4_FEW(SG_INT4_CASE)
        SG_INT4_MANY(SG_INT4_TILE)
        default: break;
    }
#undef SG_INT4_CASE
#undef SG_INT4_TILE
    return hipErrorInvalidValue;
}

template <int DT, bool ZEROS>
hipError_t launch_int4(int group, int cfg, const Int4Params& x, unsigned blocks, hipStream_t st) {
    if (group == 32) return launch_int4_group<DT, ZEROS, 32>(cfg, x, blocks, st);
    if (group == 64) return launch_int4_group<DT, ZEROS, 64>(cfg, x, blocks, st);
    return launch_int4_group<DT, ZEROS, 128>(cfg, x, blocks, st);
}

}  // namespace sg
