// ssd_recur_f32.hip -- the gated recurrence's kernels for f32 inputs (ssd_recur.h).
#include "ssd_recur.h"

namespace ssd {

const void* rec_kernel_f32(const RecurArgs& a, bool backward) { return rec_kernel<float>(a, backward); }

}  // namespace ssd
