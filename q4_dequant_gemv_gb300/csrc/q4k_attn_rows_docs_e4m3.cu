// q4k_attn_rows_docs_e4m3.cu -- the few-rows attention kernel over caches of e4m3 codes, causal calls with kv_start.
#include "q4k_attn_rows_launch.cuh"

namespace q4k {
namespace attn {
cudaError_t launch_rows_docs_e4m3(const RowsLaunch &l) { return launch_rows_type<Q4K_E4M3, 2, true>(l); }
}  // namespace attn
}  // namespace q4k
