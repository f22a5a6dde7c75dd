#include "launch_int4.hpp"

namespace sg {
template hipError_t launch_int4<DT_BF16, true>(int, int, const Int4Params&, unsigned, hipStream_t);
}
