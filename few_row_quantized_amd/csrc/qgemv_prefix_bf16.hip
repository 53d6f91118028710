// Attention over a common prefix: bfloat16 queries over a bfloat16 cache.
#include "qgemv_prefix_impl.h"

namespace qgemv {
int launch_shared_bf16(const AttendArgs &a, hipStream_t stream) { return launch_shared_t<true, false>(a, stream); }
}  // namespace qgemv
