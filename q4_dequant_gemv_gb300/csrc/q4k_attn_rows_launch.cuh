// q4k_attn_rows_launch.cuh -- host side of the few-rows attention kernel: the
// instance, its grid and its scratch.
#pragma once
#include <algorithm>

#include "q4k_attn_rows.cuh"

namespace q4k {
namespace attn {

template <int CT, int PARTS, int NT, int RG, int DP, bool TMA, bool DOCS>
static cudaError_t launch_rows_fill(const RowsLaunch &l)
{
    using Sh = RowsShared<CT, PARTS, NT, RG, DP>;
    using Sp = RowsShape<NT, RG, DP>;
    auto kern = rows_kernel<CT, PARTS, NT, RG, DP, TMA, DOCS>;
    Args a = l.args;
    constexpr int R = Sh::R;
    constexpr int kSmem = static_cast<int>(sizeof(Sh)) + 1024;   // room to align the rings to 1024 bytes
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
    CacheMaps maps;
    if (TMA && !encode_cache(&maps, a, CT, kBlock)) return cudaErrorInvalidValue;
    a.slots = static_cast<int>(static_cast<int64_t>(a.tokens) * a.group / R) + a.batch;
    const int64_t units = (static_cast<int64_t>(a.capacity) + kBlock - 1) / Sp::kUnit + 1;   // of one tile at most
    static OncePerDevice once;
    const cudaError_t attr =
        once(l.device, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
    if (attr != cudaSuccess) return attr;

    // A cluster per tile and cache head joins through its shared memory: one
    // launch, no scratch.  The split over all CTAs balances ragged lengths and a few
    // long sequences, for scratch and a join through memory.
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = Sp::kThreads;
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = l.stream;
    if (l.choice.cluster) {
        a.cluster = l.choice.cluster;
        cfg.gridDim = static_cast<unsigned>(a.slots * a.kv_heads * a.cluster);
        const Attributes at(&cfg, a.cluster, a.pdl);
        return cudaLaunchKernelEx(&cfg, kern, maps, a);
    }
    const int64_t most = static_cast<int64_t>(a.slots) * a.kv_heads * units;
    const int grid = static_cast<int>(std::min<int64_t>({most, l.sms, kMaxParts}));
    cfg.gridDim = static_cast<unsigned>(grid);
    const Attributes at(&cfg, 0, a.pdl);
    return launch_split(a, l.device, grid, R, DP, rows_shift<CT>(), l.stream,
                        [&](const Args &args) { return cudaLaunchKernelEx(&cfg, kern, maps, args); });
}

template <int CT, int PARTS, int NT, int RG, int DP, bool DOCS>
static cudaError_t launch_rows_one(const RowsLaunch &l)
{
    return l.boxes ? launch_rows_fill<CT, PARTS, NT, RG, DP, true, DOCS>(l)
                   : launch_rows_fill<CT, PARTS, NT, RG, DP, false, DOCS>(l);
}

template <int CT, int PARTS, int DP, bool DOCS>
static cudaError_t launch_rows_tiles(const RowsLaunch &l)
{
    if (l.choice.rows == 8) return launch_rows_one<CT, PARTS, 1, 1, DP, DOCS>(l);
    if constexpr (DP <= 128)
        if (l.choice.rows == 32) return launch_rows_one<CT, PARTS, 2, 2, DP, DOCS>(l);
    return launch_rows_one<CT, PARTS, 2, 1, DP, DOCS>(l);
}

// How many clusters of 1 .. kMaxCluster CTAs the GPU holds at once.  Every instance
// fills an SM with one CTA (its rings), so one stands for all.
template <int CT>
static cudaError_t rows_room(int (&n)[kMaxCluster + 1])
{
    auto kern = rows_kernel<CT, 1, 1, 1, 128, true, false>;
    constexpr int kSmem = static_cast<int>(sizeof(RowsShared<CT, 1, 1, 1, 128>)) + 1024;
    static_assert(kSmem > 227 * 1024 / 2, "one CTA per SM");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    for (int S = 1; S <= kMaxCluster && e == cudaSuccess; ++S) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = static_cast<unsigned>(1024 * S);
        cfg.blockDim = RowsShape<1, 1, 128>::kThreads;
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = S, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n[S], kern, &cfg);
    }
    return e;
}

template <int CT, int MANY, bool DOCS>
static cudaError_t launch_rows_type(const RowsLaunch &l)
{
    const int dim = l.args.dim;
    if (l.parts_many) {
        if (dim > 128) return launch_rows_tiles<CT, MANY, 256, DOCS>(l);
        return dim > 64 ? launch_rows_tiles<CT, MANY, 128, DOCS>(l) : launch_rows_tiles<CT, MANY, 64, DOCS>(l);
    }
    if (dim > 128) return launch_rows_tiles<CT, 1, 256, DOCS>(l);
    return dim > 64 ? launch_rows_tiles<CT, 1, 128, DOCS>(l) : launch_rows_tiles<CT, 1, 64, DOCS>(l);
}

}  // namespace attn
}  // namespace q4k
