// Attention kernels: bfloat16 queries over a bfloat16 cache.
#include "qgemv_attend_impl.h"

namespace qgemv {
int launch_attend_bf16(const AttendArgs &a, hipStream_t stream) { return launch_attend_t<true, false>(a, stream); }
}  // namespace qgemv
