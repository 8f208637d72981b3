// ssd_linear_e4m3_f32.hip -- the matrix product's kernels for e4m3 operands and outputs in fp32 (ssd_linear.h).
#include "ssd_linear.h"

namespace ssd {

hipError_t launch_linear_e4m3_f32(LinearArgs& a, LinearArgs* b, const LinearPlan& p, hipStream_t st) {
    return launch_linear_type<LT_E4M3_F32>(a, b, p, st);
}

}  // namespace ssd
