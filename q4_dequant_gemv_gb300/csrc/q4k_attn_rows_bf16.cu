// q4k_attn_rows_bf16.cu -- the few-rows attention kernel over bf16 caches.
#include "q4k_attn_rows_launch.cuh"

namespace q4k {
namespace attn {
cudaError_t clusters_at_once(int (&n)[kMaxCluster + 1]) { return rows_room<Q4K_BF16>(n); }
cudaError_t launch_rows_bf16(const RowsLaunch &l) { return launch_rows_type<Q4K_BF16, 3, false>(l); }
}  // namespace attn
}  // namespace q4k
