// ssd_linear_f32.hip -- the matrix product's kernels for f32 operands (ssd_linear.h).
#include "ssd_linear.h"

namespace ssd {

hipError_t launch_linear_f32(LinearArgs& a, LinearArgs* b, const LinearPlan& p, hipStream_t st) {
    return launch_linear_type<LT_F32>(a, b, p, st);
}

}  // namespace ssd
