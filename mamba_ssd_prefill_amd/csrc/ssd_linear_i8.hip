// ssd_linear_i8.hip -- the matrix product's kernels for i8 operands (ssd_linear.h).
#include "ssd_linear.h"

namespace ssd {

hipError_t launch_linear_i8(LinearArgs& a, LinearArgs* b, const LinearPlan& p, hipStream_t st) {
    return launch_linear_type<LT_I8>(a, b, p, st);
}

}  // namespace ssd
