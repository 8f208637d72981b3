// ssd_linear_f16.hip -- the matrix product's kernels for f16 operands (ssd_linear.h).
#include "ssd_linear.h"

namespace ssd {

hipError_t launch_linear_f16(LinearArgs& a, LinearArgs* b, const LinearPlan& p, hipStream_t st) {
    return launch_linear_type<LT_F16>(a, b, p, st);
}

}  // namespace ssd
