// Attention over a common prefix: bfloat16 queries over an E4M3 cache.
#include "qgemv_prefix_impl.h"

namespace qgemv {
int launch_shared_bf16_e4m3(const AttendArgs &a, hipStream_t stream) { return launch_shared_t<true, true>(a, stream); }
}  // namespace qgemv
