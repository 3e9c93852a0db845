// q4k_attn_chunk_launch.cuh -- host side of the many-rows attention kernel: the
// variant by sizes, its grid and its scratch.
#pragma once
#include <algorithm>

#include "q4k_attn_chunk.cuh"

namespace q4k {
namespace attn {

template <int CT, int DP, int MODE>
static cudaError_t launch_chunk_one(const ChunkLaunch &l)
{
    using Sh = ChunkShared<DP>;
    auto kern = chunk_kernel<CT, DP, MODE>;
    Args a = l.args;
    constexpr int R = kChunkRows;
    constexpr int kSmem = static_cast<int>(sizeof(Sh)) + 1024;   // room to align the tiles to 1024 bytes
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
    int box = 128;
    while (a.page_size % box) box /= 2;
    CacheMaps maps;
    CUtensorMap qmap;
    const int tokens = R / a.group;   // of a tile
    if (!encode_cache(&maps, a, CT, box) || !encode_queries(&qmap, a, CT, tokens)) return cudaErrorInvalidValue;
    a.slots = a.tokens / tokens + a.batch;
    const int64_t units = a.capacity / kChunkKeys + 1;
    const int64_t most = static_cast<int64_t>(a.slots) * a.kv_heads * units;
    const int grid = static_cast<int>(std::min<int64_t>({most, l.sms, kMaxParts}));
    static OncePerDevice once;
    const cudaError_t attr =
        once(l.device, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
    if (attr != cudaSuccess) return attr;
    return launch_split(a, l.device, grid, R, DP, chunk_shift<CT>(), l.stream, [&](const Args &args) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = kChunkThreads;
        cfg.dynamicSmemBytes = kSmem;
        cfg.stream = l.stream;
        const Attributes at(&cfg, 0, args.pdl);
        return cudaLaunchKernelEx(&cfg, kern, maps, qmap, args, box);
    });
}

template <int CT, int DP>
static cudaError_t launch_chunk_mode(const ChunkLaunch &l)
{
    switch ((l.args.softcap > 0.0f ? 1 : 0) | (l.args.slopes ? 2 : 0) | (l.args.docs() ? 4 : 0)) {
        case 0: return launch_chunk_one<CT, DP, 0>(l);
        case 1: return launch_chunk_one<CT, DP, 1>(l);
        case 2: return launch_chunk_one<CT, DP, 2>(l);
        case 3: return launch_chunk_one<CT, DP, 3>(l);
        case 4: return launch_chunk_one<CT, DP, 4>(l);
        case 5: return launch_chunk_one<CT, DP, 5>(l);
        case 6: return launch_chunk_one<CT, DP, 6>(l);
        default: return launch_chunk_one<CT, DP, 7>(l);
    }
}

template <int CT>
static cudaError_t launch_chunk_type(const ChunkLaunch &l)
{
    return l.args.dim > 64 ? launch_chunk_mode<CT, 128>(l) : launch_chunk_mode<CT, 64>(l);
}

}  // namespace attn
}  // namespace q4k
