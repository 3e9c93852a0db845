// q4k_attn_chunk_wide.cu -- the many-rows attention kernel over widened 8-bit caches.
#include "q4k_attn_chunk_launch.cuh"

namespace q4k {
namespace attn {
cudaError_t launch_chunk_wide(const ChunkLaunch &l) { return launch_chunk_type<Q4K_F16, 8>(l); }
}  // namespace attn
}  // namespace q4k
