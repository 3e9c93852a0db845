// q4k_attn_rows_f16.cu -- the few-rows attention kernel over fp16 caches.
#include "q4k_attn_rows_launch.cuh"

namespace q4k {
namespace attn {
cudaError_t launch_rows_f16(const RowsLaunch &l) { return launch_rows_type<Q4K_F16, 2, false>(l); }
}  // namespace attn
}  // namespace q4k
