// q4k_attn_rows_launch.cuh -- host side of the few-rows attention kernel: the
// variant by sizes, its grid and its scratch.
#pragma once
#include <algorithm>

#include "q4k_attn_rows.cuh"

namespace q4k {
namespace attn {

template <int CT, int PARTS, int NT, int DP>
static cudaError_t launch_rows_one(const RowsLaunch &l)
{
    using Sh = RowsShared<CT, PARTS, NT, DP>;
    auto kern = rows_kernel<CT, PARTS, NT, DP>;
    constexpr int per_sm = (NT == 1 && DP <= 128) ? 2 : 1;
    Args a = l.args;
    constexpr int R = Sh::R;
    a.slots = static_cast<int>(static_cast<int64_t>(a.tokens) * a.group / R) + a.batch;
    const int64_t units = (a.capacity + 15) / kRowsUnit + 1;   // of one tile at most
    const int64_t most = static_cast<int64_t>(a.slots) * a.kv_heads * units;
    const int grid = static_cast<int>(std::min<int64_t>(most, static_cast<int64_t>(l.sms) * per_sm));
    static const cudaError_t attr =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Sh)));
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
    kern<<<grid, kRowsThreads, sizeof(Sh), l.stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (scratch) {
        const cudaError_t f = cudaFreeAsync(scratch, l.stream);
        if (e == cudaSuccess) e = f;
    }
    return e;
}

template <int CT, int MANY>
static cudaError_t launch_rows_type(const RowsLaunch &l)
{
    // 16 query rows where sequences bring more than 8 per cache head: half the
    // reads of the cache
    const bool two = static_cast<int64_t>(l.args.tokens) * l.args.group > 8 * static_cast<int64_t>(l.args.batch);
    const int dim = l.args.dim;
    if (l.parts_many) {
        if (dim > 128) return launch_rows_one<CT, MANY, 1, 256>(l);
        if (dim > 64) return two ? launch_rows_one<CT, MANY, 2, 128>(l) : launch_rows_one<CT, MANY, 1, 128>(l);
        return two ? launch_rows_one<CT, MANY, 2, 64>(l) : launch_rows_one<CT, MANY, 1, 64>(l);
    }
    if (dim > 128) return launch_rows_one<CT, 1, 1, 256>(l);
    if (dim > 64) return two ? launch_rows_one<CT, 1, 2, 128>(l) : launch_rows_one<CT, 1, 1, 128>(l);
    return two ? launch_rows_one<CT, 1, 2, 64>(l) : launch_rows_one<CT, 1, 1, 64>(l);
}

}  // namespace attn
}  // namespace q4k
