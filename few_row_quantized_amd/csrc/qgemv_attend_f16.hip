// Attention kernels: float16 queries over a float16 cache.
#include "qgemv_attend_impl.h"

namespace qgemv {
int launch_attend_f16(const AttendArgs &a, hipStream_t stream) { return launch_attend_t<false, false>(a, stream); }
}  // namespace qgemv
