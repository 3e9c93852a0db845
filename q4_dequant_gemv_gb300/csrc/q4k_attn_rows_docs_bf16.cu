// q4k_attn_rows_docs_bf16.cu -- the few-rows attention kernel over a bf16 cache, causal calls with kv_start.
#include "q4k_attn_rows_launch.cuh"

namespace q4k {
namespace attn {
cudaError_t launch_rows_docs_bf16(const RowsLaunch &l) { return launch_rows_type<Q4K_BF16, 3, true>(l); }
}  // namespace attn
}  // namespace q4k
