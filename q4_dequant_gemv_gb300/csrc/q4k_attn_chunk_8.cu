// q4k_attn_chunk_8.cu -- the many-rows attention kernel over 8-bit caches (codes of either type).
#include "q4k_attn_chunk_launch.cuh"

namespace q4k {
namespace attn {
cudaError_t launch_chunk_8(const ChunkLaunch &l) { return launch_chunk_type<Q4K_I8>(l); }
}  // namespace attn
}  // namespace q4k
