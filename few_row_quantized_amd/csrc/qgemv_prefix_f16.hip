// Attention over a common prefix: float16 queries over a float16 cache.
#include "qgemv_prefix_impl.h"

namespace qgemv {
int launch_shared_f16(const AttendArgs &a, hipStream_t stream) { return launch_shared_t<false, false>(a, stream); }
}  // namespace qgemv
