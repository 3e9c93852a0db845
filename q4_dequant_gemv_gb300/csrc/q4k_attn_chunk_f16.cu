// q4k_attn_chunk_f16.cu -- the many-rows attention kernel over fp16 caches.
#include "q4k_attn_chunk_launch.cuh"

namespace q4k {
namespace attn {
cudaError_t launch_chunk_f16(const ChunkLaunch &l) { return launch_chunk_type<Q4K_F16>(l); }
}  // namespace attn
}  // namespace q4k
