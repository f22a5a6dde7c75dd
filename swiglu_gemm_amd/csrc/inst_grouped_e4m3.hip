// e4m3 instantiations of the grouped GEMM launchers.
#include "launch_grouped.hpp"
namespace sg {
template hipError_t launch_grouped<DT_E4M3>(int, bool, bool, int, const GroupedParams&, unsigned, hipStream_t);
}
