// Attention kernels: float16 queries over an E4M3 cache.
#include "qgemv_attend_impl.h"

namespace qgemv {
int launch_attend_f16_e4m3(const AttendArgs &a, hipStream_t stream) { return launch_attend_t<false, true>(a, stream); }
}  // namespace qgemv
