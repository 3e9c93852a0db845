// q4k_attn_chunk_bf16.cu -- the many-rows attention kernel over bf16 caches.
#include "q4k_attn_chunk_launch.cuh"

namespace q4k {
namespace attn {
cudaError_t launch_chunk_bf16(const ChunkLaunch &l) { return launch_chunk_type<Q4K_BF16>(l); }
}  // namespace attn
}  // namespace q4k
