// q4k_attn_rows_launch.cuh -- host side of the few-rows attention kernel: the
// variant by sizes, its grid and its scratch.
#pragma once
#include <algorithm>

#include "q4k_attn_rows.cuh"

namespace q4k {
namespace attn {

template <int CT, int PARTS, int NT, int DP, bool TMA>
static cudaError_t launch_rows_fill(const RowsLaunch &l)
{
    using Sh = RowsShared<CT, PARTS, NT, DP>;
    using Sp = RowsShape<DP>;
    auto kern = rows_kernel<CT, PARTS, NT, DP, TMA>;
    Args a = l.args;
    constexpr int R = Sh::R;
    constexpr int kSmem = static_cast<int>(sizeof(Sh)) + 1024;   // room to align the rings to 1024 bytes
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
    CacheMaps maps;
    if (TMA && !encode_cache(&maps, a, CT, kBlock)) return cudaErrorInvalidValue;
    a.slots = static_cast<int>(static_cast<int64_t>(a.tokens) * a.group / R) + a.batch;
    const int64_t units = (a.capacity + kBlock - 1) / Sp::kUnit + 1;   // of one tile at most
    const int64_t most = static_cast<int64_t>(a.slots) * a.kv_heads * units;
    const int grid = static_cast<int>(std::min<int64_t>(most, l.sms));
    static const cudaError_t attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (attr != cudaSuccess) return attr;
    const size_t head = (grid * sizeof(unsigned int) + 255) / 256 * 256;
    void *scratch = nullptr;
    if (units > 1) {
        const size_t bytes = head + static_cast<size_t>(grid) * 2 * R * (DP + 2) * sizeof(float);
        cudaError_t e = cudaMallocAsync(&scratch, bytes, l.stream);
        if (e != cudaSuccess) return e;
        e = cudaMemsetAsync(scratch, 0, grid * sizeof(unsigned int), l.stream);
        if (e != cudaSuccess) {
            (void)cudaFreeAsync(scratch, l.stream);
            return e;
        }
        a.ticket = static_cast<unsigned int *>(scratch);
        a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(scratch) + head);
    }
    kern<<<grid, Sp::kThreads, kSmem, l.stream>>>(maps, a);
    cudaError_t e = cudaGetLastError();
    if (scratch) {
        const cudaError_t f = cudaFreeAsync(scratch, l.stream);
        if (e == cudaSuccess) e = f;
    }
    return e;
}

template <int CT, int PARTS, int NT, int DP>
static cudaError_t launch_rows_one(const RowsLaunch &l)
{
    return l.boxes ? launch_rows_fill<CT, PARTS, NT, DP, true>(l) : launch_rows_fill<CT, PARTS, NT, DP, false>(l);
}

template <int CT, int PARTS, int DP>
static cudaError_t launch_rows_tiles(const RowsLaunch &l)
{
    // the smallest tile that holds the rows an average sequence brings (fewer
    // reads of the cache), 8 to 32; dim > 128 leaves registers for 16
    const int64_t rows = static_cast<int64_t>(l.args.tokens) * l.args.group, batch = l.args.batch;
    if (rows <= 8 * batch) return launch_rows_one<CT, PARTS, 1, DP>(l);
    if constexpr (DP <= 128)
        if (rows > 16 * batch) return launch_rows_one<CT, PARTS, 4, DP>(l);
    return launch_rows_one<CT, PARTS, 2, DP>(l);
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
