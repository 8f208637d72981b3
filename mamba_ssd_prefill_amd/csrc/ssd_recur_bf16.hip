// ssd_recur_bf16.hip -- the gated recurrence's kernels for bf16 inputs (ssd_recur.h).
#include "ssd_recur.h"

namespace ssd {

const void* rec_kernel_bf16(const RecurArgs& a, bool backward) { return rec_kernel<__bf16>(a, backward); }

}  // namespace ssd
