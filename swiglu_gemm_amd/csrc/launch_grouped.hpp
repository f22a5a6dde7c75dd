// launch_grouped.hpp -- launchers of the grouped kernels for one operand type, each type
// instantiated in its own translation unit (inst_grouped_*.hip).
#pragma once

#include "grouped.hpp"
#include "grouped_dma.hpp"

namespace sg {

template <int DT, bool TA, bool TB, int EPI>
hipError_t launch_grouped_epi(int cfg, const GroupedParams& q, unsigned blocks, hipStream_t st) {
    if (cfg < 0) {
        hipLaunchKernelGGL((grouped_any_kernel<DT, TA, TB, EPI>), dim3(blocks), dim3(256), 0, st,
                           q);
        return hipGetLastError();
    }
#define SG_GCASE(ID, BM, BN, BK, S, WM, WN)                                                   \
    case ID:                                                                                  \
        hipLaunchKernelGGL((grouped_dma_kernel<DT, TA, TB, EPI, BM, BN, BK, S, WM, WN>),      \
                           dim3(blocks), dim3(64 * WM * WN), 0, st, q);                       \
        return hipGetLastError();
    if constexpr (DT == DT_E4M3) {
        switch (cfg) {
            SG_GROUPED_8(SG_GCASE)
            default: return hipErrorInvalidValue;
        }
    } else if constexpr (TA) {
        switch (cfg) {
            SG_GROUPED_DEPTH(SG_GCASE)
            default: return hipErrorInvalidValue;
        }
    } else {
        switch (cfg) {
            SG_GROUPED_16(SG_GCASE)
            default: return hipErrorInvalidValue;
        }
    }
#undef SG_GCASE
}

template <int DT>
hipError_t launch_grouped(int epi, bool ta, bool tb, int cfg, const GroupedParams& q,
                          unsigned blocks, hipStream_t st) {
    if (ta) {
        if constexpr (DT != DT_E4M3) {
            if (epi == EPI_GEMM)
                return launch_grouped_epi<DT, true, false, EPI_GEMM>(cfg, q, blocks, st);
            if (epi == EPI_GEMM_F32)
                return launch_grouped_epi<DT, true, false, EPI_GEMM_F32>(cfg, q, blocks, st);
        }
        return hipErrorInvalidValue;
    }
    if (epi == EPI_GEMM)
        return tb ? launch_grouped_epi<DT, false, true, EPI_GEMM>(cfg, q, blocks, st)
                  : launch_grouped_epi<DT, false, false, EPI_GEMM>(cfg, q, blocks, st);
    if (epi == EPI_SWIGLU)
        return launch_grouped_epi<DT, false, false, EPI_SWIGLU>(cfg, q, blocks, st);
    if constexpr (DT != DT_E4M3) {
        if (epi == EPI_SWIGLU_BWD)
            return launch_grouped_epi<DT, false, false, EPI_SWIGLU_BWD>(cfg, q, blocks, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace sg
