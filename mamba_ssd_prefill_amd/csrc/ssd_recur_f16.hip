// ssd_recur_f16.hip -- the gated recurrence's kernels for f16 inputs (ssd_recur.h).
#include "ssd_recur.h"

namespace ssd {

const void* rec_kernel_f16(const RecurArgs& a, bool backward) { return rec_kernel<_Float16>(a, backward); }

}  // namespace ssd
