// q4k_attn_rows_launch.cuh -- host side of the few-rows attention kernel: the
// variant by sizes, its grid and its scratch.
#pragma once
#include <algorithm>

#include "q4k_attn_rows.cuh"

namespace q4k {
namespace attn {

constexpr double kSplitCost = 18.0;

// How many clusters of S CTAs of a kernel the GPU holds at once.
struct Together {
    int n[kMaxCluster + 1];
};

template <class Kernel>
static Together clusters_at_once(Kernel kern, int threads, int smem, int sms)
{
    Together t{};
    t.n[1] = sms;
    for (int S = 2; S <= kMaxCluster; ++S) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = static_cast<unsigned>(sms * S);
        cfg.blockDim = threads;
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = S, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&t.n[S], kern, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            t.n[S] = 0;
        }
    }
    return t;
}

template <int CT, int PARTS, int NT, int RG, int DP, bool TMA>
static cudaError_t launch_rows_fill(const RowsLaunch &l)
{
    using Sh = RowsShared<CT, PARTS, NT, RG, DP>;
    using Sp = RowsShape<NT, RG, DP>;
    auto kern = rows_kernel<CT, PARTS, NT, RG, DP, TMA>;
    Args a = l.args;
    constexpr int R = Sh::R;
    constexpr int kSmem = static_cast<int>(sizeof(Sh)) + 1024;   // room to align the rings to 1024 bytes
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
    CacheMaps maps;
    if (TMA && !encode_cache(&maps, a, CT, kBlock)) return cudaErrorInvalidValue;
    a.slots = static_cast<int>(static_cast<int64_t>(a.tokens) * a.group / R) + a.batch;
    const int64_t units = (static_cast<int64_t>(a.capacity) + kBlock - 1) / Sp::kUnit + 1;   // of one tile at most
    static const cudaError_t attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (attr != cudaSuccess) return attr;

    // A cluster of S CTAs per tile and cache head joins through its shared
    // memory: one launch, no scratch.  The split over all CTAs balances ragged
    // lengths and a few long sequences, but its scratch and the join through memory
    // cost about kSplitCost units of one CTA's time.
    const int64_t items = a.kv_heads * std::max<int64_t>(a.batch, (static_cast<int64_t>(a.tokens) * a.group + R - 1) / R);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = Sp::kThreads;
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = l.stream;
    // the cluster size that ends soonest: waves of clusters times units of a rank
    static const Together room = clusters_at_once(kern, Sp::kThreads, kSmem, l.sms);
    int S = 1;
    int64_t by_cluster = INT64_MAX;
    for (int c = 1; c <= kMaxCluster && c <= units; ++c) {
        if (room.n[c] < 1) continue;
        const int64_t cost = (items + room.n[c] - 1) / room.n[c] * ((units + c - 1) / c);
        if (cost < by_cluster) by_cluster = cost, S = c;
    }
    const double by_split = static_cast<double>(items) * units / l.sms;
    if (static_cast<double>(by_cluster) <= by_split + kSplitCost && static_cast<int64_t>(a.slots) * a.kv_heads * S < (1 << 24)) {
        a.cluster = S;
        cfg.gridDim = static_cast<unsigned>(a.slots * a.kv_heads * S);
        const Attributes at(&cfg, S, a.pdl);
        return cudaLaunchKernelEx(&cfg, kern, maps, a);
    }
    const int64_t most = static_cast<int64_t>(a.slots) * a.kv_heads * units;
    const int grid = static_cast<int>(std::min<int64_t>({most, l.sms, kMaxParts}));
    cfg.gridDim = static_cast<unsigned>(grid);
    const Attributes at(&cfg, 0, a.pdl);
    return launch_split(a, grid, R, DP, rows_shift<CT>(), l.stream,
                        [&](const Args &args) { return cudaLaunchKernelEx(&cfg, kern, maps, args); });
}

template <int CT, int PARTS, int NT, int RG, int DP>
static cudaError_t launch_rows_one(const RowsLaunch &l)
{
    return l.boxes ? launch_rows_fill<CT, PARTS, NT, RG, DP, true>(l) : launch_rows_fill<CT, PARTS, NT, RG, DP, false>(l);
}

template <int CT, int PARTS, int DP>
static cudaError_t launch_rows_tiles(const RowsLaunch &l)
{
    // the smallest tile that holds a sequence's rows (a second tile reads its
    // keys again): those of one token where there are as many tokens as
    // sequences, all of a single sequence, else half as many again as the average.
    // dim > 128 leaves registers for 16.
    const int64_t batch = l.args.batch, all = static_cast<int64_t>(l.args.tokens) * l.args.group;
    const int64_t rows = l.args.tokens == batch ? l.args.group : batch == 1 ? all : (3 * all + 2 * batch - 1) / (2 * batch);
    if (rows <= 8) return launch_rows_one<CT, PARTS, 1, 1, DP>(l);
    if constexpr (DP <= 128) {
        if (rows > 32) return launch_rows_one<CT, PARTS, 3, 2, DP>(l);
        if (rows > 16) return launch_rows_one<CT, PARTS, 2, 2, DP>(l);
    }
    return launch_rows_one<CT, PARTS, 2, 1, DP>(l);
}

template <int CT, int MANY>
static cudaError_t launch_rows_type(const RowsLaunch &l)
{
    const int dim = l.args.dim;
    if (l.parts_many) {
        if (dim > 128) return launch_rows_tiles<CT, MANY, 256>(l);
        return dim > 64 ? launch_rows_tiles<CT, MANY, 128>(l) : launch_rows_tiles<CT, MANY, 64>(l);
    }
    if (dim > 128) return launch_rows_tiles<CT, 1, 256>(l);
    return dim > 64 ? launch_rows_tiles<CT, 1, 128>(l) : launch_rows_tiles<CT, 1, 64>(l);
}

}  // namespace attn
}  // namespace q4k
