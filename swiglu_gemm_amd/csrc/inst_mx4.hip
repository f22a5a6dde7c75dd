// The 4-bit product's kernels.
#include "mx4_dma.hpp"

namespace sg {

template <int DT_OUT, int EPI>
static hipError_t launch_mx4_epi(int cfg, const MxParams& x, unsigned blocks, hipStream_t st) {
#define SG_MXCASE(ID, BM, BN, S, WM, WN)                                                       \
    case ID:                                                                                   \
        hipLaunchKernelGGL((mx_dma_kernel<DT_OUT, EPI, BM, BN, S, WM, WN>), dim3(blocks),      \
                           dim3(64 * WM * WN), 0, st, x);                                      \
        return hipGetLastError();
    switch (cfg) {
        SG_MX_CONFIGS(SG_MXCASE)
        default: break;
    }
#undef SG_MXCASE
    return hipErrorInvalidValue;
}

hipError_t launch_mx4(int epi, int dt, int cfg, const MxParams& x, unsigned blocks,
                      hipStream_t st) {
    if (epi == EPI_GEMM_F32) return launch_mx4_epi<DT_BF16, EPI_GEMM_F32>(cfg, x, blocks, st);
    if (epi == EPI_GEMM)
        return dt == DT_F16 ? launch_mx4_epi<DT_F16, EPI_GEMM>(cfg, x, blocks, st)
                            : launch_mx4_epi<DT_BF16, EPI_GEMM>(cfg, x, blocks, st);
    if (epi == EPI_SWIGLU)
        return dt == DT_F16 ? launch_mx4_epi<DT_F16, EPI_SWIGLU>(cfg, x, blocks, st)
                            : launch_mx4_epi<DT_BF16, EPI_SWIGLU>(cfg, x, blocks, st);
    return hipErrorInvalidValue;
}

}  // namespace sg
