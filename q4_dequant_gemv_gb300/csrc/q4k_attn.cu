// q4k_attn.cu -- q4k_paged_attention: argument checks and the choice of kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/q4k.h"
#include "q4k_attn_chunk.cuh"
#include "q4k_attn_plan.h"
#include "q4k_attn_rows.cuh"
#include "q4k_internal.h"

namespace q4k {

__device__ unsigned int g_attn_error = 0;   // bit 2: an index outside its buffer, bit 3: a bounded wait timed out

unsigned int read_attn_error()
{
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_error, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    return v;
}

bool clear_attn_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_attn_error, &z, sizeof(z)) == cudaSuccess;
}

// Address of the error word on a device.
static cudaError_t error_word(int dev, unsigned int **p)
{
    static unsigned int *at[attn::kDevices];
    static attn::OncePerDevice once;
    const cudaError_t e = once(dev, [&] { return cudaGetSymbolAddress(reinterpret_cast<void **>(&at[dev]), g_attn_error); });
    *p = at[dev];
    return e;
}

namespace attn {

// Calls of this thread that a capture under way on another stream, or on the
// call's own, does not concern: creating a pool is refused during a capture
// otherwise, and ends it.
struct BesideCaptures {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    BesideCaptures() { (void)cudaThreadExchangeStreamCaptureMode(&mode); }
    ~BesideCaptures() { (void)cudaThreadExchangeStreamCaptureMode(&mode); }
};

// Scratch comes from a pool of the library's own, one per device, that keeps its
// memory: the default pool gives it back to the system whenever the program
// synchronises, and the next call then waits 250 us for it.
cudaError_t take_scratch(int dev, void **p, size_t bytes, cudaStream_t stream)
{
    static cudaMemPool_t pools[kDevices];
    static OncePerDevice once;
    const cudaError_t e = once(dev, [&] {
        const BesideCaptures beside;   // (a first call may be a captured one)
        cudaMemPoolProps props = {};
        props.allocType = cudaMemAllocationTypePinned;
        props.location.type = cudaMemLocationTypeDevice;
        props.location.id = dev;
        cudaMemPool_t made = nullptr;
        cudaError_t bad = cudaMemPoolCreate(&made, &props);
        if (bad != cudaSuccess) return bad;
        cuuint64_t keep = UINT64_MAX;
        bad = cudaMemPoolSetAttribute(made, cudaMemPoolAttrReleaseThreshold, &keep);
        if (bad != cudaSuccess) (void)cudaMemPoolDestroy(made);
        else pools[dev] = made;
        return bad;
    });
    return e == cudaSuccess ? cudaMallocFromPoolAsync(p, bytes, pools[dev], stream) : e;
}

// Clusters of each size that a device holds at once.
static cudaError_t room_of(int dev, const int (**room)[kMaxCluster + 1])
{
    static int n[kDevices][kMaxCluster + 1];
    static OncePerDevice once;
    *room = &n[dev];
    return once(dev, [&] { return clusters_at_once(n[dev]); });
}

bool encode_cache(CacheMaps *maps, const Args &a, int type, int box)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    auto one = [&](CUtensorMap *map, const void *base, int64_t page, int64_t slot, int64_t head) {
        // a stride that no index uses may be anything; the encoder wants a legal one
        const int64_t row = (a.dim + 7) / 8 * 8;
        if (a.kv_heads == 1) head = row;
        if (a.pages == 1) page = row;
        cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.dim), static_cast<cuuint64_t>(a.page_size),
                              static_cast<cuuint64_t>(a.kv_heads), static_cast<cuuint64_t>(a.pages)};
        cuuint64_t strides[3] = {static_cast<cuuint64_t>(slot) * 2, static_cast<cuuint64_t>(head) * 2,
                                 static_cast<cuuint64_t>(page) * 2};
        cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), 1, 1}, steps[4] = {1, 1, 1, 1};
        return enc(map, type == Q4K_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                   const_cast<void *>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return one(&maps->k, a.k, a.k_page, a.k_slot, a.k_head) && one(&maps->v, a.v, a.v_page, a.v_slot, a.v_head);
}

bool encode_queries(CUtensorMap *map, const Args &a, int type, int tokens)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const int64_t row = (a.dim + 7) / 8 * 8;
    const int64_t token = a.tokens == 1 ? row : a.q_token, head = a.heads == 1 ? row : a.q_head;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.dim), static_cast<cuuint64_t>(a.heads),
                          static_cast<cuuint64_t>(a.tokens)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(token) * 2};
    cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(a.group), static_cast<cuuint32_t>(tokens)}, steps[3] = {1, 1, 1};
    return enc(map, type == Q4K_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void *>(a.q), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A statistic of `slab` rows of up to `grid` parts, in whole float4.
__host__ __device__ __forceinline__ int join_floats(int slab, int grid) { return (slab * grid + 3) & ~3; }

// Adds the parts of split tiles: blockIdx.x = the CTA in whose share the tile
// begins, blockIdx.y = `slab` of its rows.  Bound by trips to memory, so there are
// three: the tile, all parts' statistics (they become weights in shared memory), then
// column quads.  A slab of a few rows has fewer quads than the CTA has threads: groups
// of threads take a range of the parts each, and their sums are added in order.  One
// CTA a tile of 8 rows, a part after the other, cost 0.4 us a part: 2 heads of 30000
// positions 28.6 us, now 16.8; 8 heads of 131072 93, now 90.  Launched as the first
// kernel's programmatic dependent; its shared memory is sized by the call, so that
// after the few-rows kernel it is already there, beside that kernel's rings.
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Args a, int R, int slab, int width, float shift)
{
    extern __shared__ __align__(16) float s_stats[];
    float *s_m = s_stats, *s_l = s_stats + join_floats(slab, gridDim.x);   // (s_l: later the sums of thread groups)
    __shared__ float s_max[kJoinRows], s_sum[kJoinRows];
    pdl_wait();
    const int4 t0 = __ldcg(reinterpret_cast<const int4 *>(a.joint + blockIdx.x));
    const int2 t1 = __ldcg(reinterpret_cast<const int2 *>(a.joint + blockIdx.x) + 2);
    const Joint t{t0.x, t0.y, t0.z, t0.w, t1.x, t1.y};
    const int r0 = blockIdx.y * slab, rows = min(min(R - r0, slab), t.rows - r0);
    if (rows <= 0) return;
    const int tid = threadIdx.x, parts = t.c1 - t.c0 + 1;
    const int64_t size = static_cast<int64_t>(R) * (width + 2);
    const float *first = a.part + part_slot(t.c0, true) * size + r0, *rest = a.part + part_slot(t.c0, false) * size + r0;
    auto slot = [&](int q) { return q == 0 ? first : rest + 2 * q * size; };
#pragma unroll 4
    for (int i = tid; i < parts * rows; i += kJoinThreads) {
        const int q = i / rows, r = i - q * rows;
        const float *p = slot(q) + R * width + r;
        s_m[i] = __ldcg(p), s_l[i] = __ldcg(p + R);
    }
    __syncthreads();
    if (parts <= 8 && rows > kJoinThreads / 32) {
        if (tid < rows) {
            float mx = -INFINITY, ls = 0.0f;
            for (int q = 0; q < parts; ++q) mx = fmaxf(mx, s_m[q * rows + tid]);
            for (int q = 0; q < parts; ++q) {
                const float f = weight(s_m[q * rows + tid], mx);
                s_m[q * rows + tid] = f;
                ls += f * s_l[q * rows + tid];
            }
            s_max[tid] = mx, s_sum[tid] = ls;
        }
    } else {
        for (int r = tid >> 5; r < rows; r += kJoinThreads / 32) {
            float mx = -INFINITY, ls = 0.0f;
            for (int q = tid & 31; q < parts; q += 32) mx = fmaxf(mx, s_m[q * rows + r]);
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            for (int q = tid & 31; q < parts; q += 32) {
                const float f = weight(s_m[q * rows + r], mx);
                s_m[q * rows + r] = f;
                ls += f * s_l[q * rows + r];
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
            if ((tid & 31) == 0) s_max[r] = mx, s_sum[r] = ls;
        }
    }
    __syncthreads();
    const int quads = rows * (a.dim / 4);
    auto finish = [&](int r, int c, float4 v) {
        const int row = t.first + r0 + r, tok = row / a.group;
        finish_row(a, t.tok0 + tok, t.head * a.group + row - tok * a.group, 4 * c, v, s_max[r], s_sum[r], shift);
    };
    if (quads <= kJoinThreads) {
        // groups of threads take a range of the parts each, eight loads on their way at once
        const int groups = max(1, min(kJoinThreads / quads, (parts + 3) / 4));
        const int g = tid / quads, i = tid - g * quads, c = i / rows, r = i - c * rows;
        float4 v = make_float4(0, 0, 0, 0);
        if (g < groups) {
            const int q1 = parts * (g + 1) / groups;
            for (int q = parts * g / groups; q < q1; q += 8) {
                float4 x[8];
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    x[d] = q + d < q1 ? __ldcg(reinterpret_cast<const float4 *>(slot(q + d) - r0) + r0 + c * R + r)
                                      : make_float4(0, 0, 0, 0);
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    const float f = q + d < q1 ? s_m[(q + d) * rows + r] : 0.0f;
                    v.x += f * x[d].x, v.y += f * x[d].y, v.z += f * x[d].z, v.w += f * x[d].w;
                }
            }
        }
        float4 *s_v = reinterpret_cast<float4 *>(s_l);
        s_v[tid] = v;
        __syncthreads();
        if (g) return;
        for (int k = 1; k < groups; ++k) {
            const float4 x = s_v[k * quads + i];
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        finish(r, c, v);
        return;
    }
    // else a thread takes PER quads i, i + kJoinThreads, .. (neighbouring threads on neighbouring
    // rows): a few parts: more quads in flight, many: more parts
    auto several = [&](auto per_c, auto deep_c) {
        constexpr int PER = decltype(per_c)::value, DEEP = decltype(deep_c)::value;
        for (int i = tid; i < quads; i += PER * kJoinThreads) {
            float4 v[PER];
            int c[PER], r[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) {   // (quads past the end are read again, not stored)
                const int n = i + k * kJoinThreads < quads ? i + k * kJoinThreads : i;
                c[k] = n / rows, r[k] = n - c[k] * rows;
                v[k] = make_float4(0, 0, 0, 0);
            }
#pragma unroll DEEP
            for (int q = 0; q < parts; ++q) {
                const float4 *p = reinterpret_cast<const float4 *>(slot(q) - r0) + r0;
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const float4 x = __ldcg(p + c[k] * R + r[k]);
                    const float f = s_m[q * rows + r[k]];
                    v[k].x += f * x.x, v[k].y += f * x.y, v[k].z += f * x.z, v[k].w += f * x.w;
                }
            }
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (i + k * kJoinThreads < quads) finish(r[k], c[k], v[k]);
        }
    };
    if (parts <= 4) several(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
    else several(std::integral_constant<int, 2>{}, std::integral_constant<int, 8>{});
}

cudaError_t launch_join(const Args &a, int grid, int R, int width, float shift, cudaStream_t stream)
{
    // Few large tiles have many parts each (16 tokens over 14336: 27.6 us with slabs of 16
    // rows, 31.9 of 32), many have two or three (three chunks of 512 tokens: 84 and 81).
    const int slab = R <= 32 ? 2 : static_cast<int64_t>(a.slots) * a.kv_heads * 3 <= grid ? kJoinRows / 2 : kJoinRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, (R + slab - 1) / slab);
    cfg.blockDim = kJoinThreads;
    const int floats = join_floats(slab, grid);
    cfg.dynamicSmemBytes = 4 * floats + std::max<int>(4 * floats, 16 * kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel, a, R, slab, width, shift);
}

}  // namespace attn

q4k_status paged_attention_impl(const q4k_paged_cache *c, const q4k_attention_args *a, void *stream)
{
    q4k_status st = check_cache(c);
    if (st == Q4K_ERR_INVALID_ARG || !a) return Q4K_ERR_INVALID_ARG;
    const q4k_paged_cache used = with_used_strides(*c);
    c = &used;
    auto type_ok = [](int t) { return t == Q4K_F32 || t == Q4K_F16 || t == Q4K_BF16; };
    if (c->dim % 8 || c->dim > 256 || a->q_heads < 1 || a->q_heads > 65536 || a->q_heads % c->heads ||
        !type_ok(a->q_type) || !type_ok(a->out_type) || (a->causal & ~1) || a->window < 0 ||
        !std::isfinite(a->scale) || !std::isfinite(a->softcap) || a->softcap < 0.0f ||
        c->tokens * a->q_heads > 0x7FFFFFFF || (a->flags & ~(Q4K_FLAG_PDL | Q4K_FLAG_TEST_STALL | Q4K_FLAG_ATTN_FORM(7))))
        return Q4K_ERR_INVALID_ARG;
    const bool some = c->tokens > 0 && c->batch > 0;
    if (some && (!a->q || !a->out)) return Q4K_ERR_INVALID_ARG;
    if (st != Q4K_OK) return st;
    auto off16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; };
    auto off4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
    const int64_t qn = a->q_type == Q4K_F32 ? 4 : 8, on = a->out_type == Q4K_F32 ? 4 : 8;
    const int64_t q_token = used_stride(a->q_token_stride, c->tokens), q_head = used_stride(a->q_head_stride, a->q_heads);
    const int64_t out_token = used_stride(a->out_token_stride, c->tokens), out_head = used_stride(a->out_head_stride, a->q_heads);
    if (off16(c->k) || off16(c->v) || off16(a->q) || off16(a->out) || off4(a->lse) || off4(a->slopes) ||
        off4(a->prefix_len) || off4(a->kv_start) || c->k_page_stride % 8 || c->k_slot_stride % 8 ||
        c->k_head_stride % 8 || c->v_page_stride % 8 || c->v_slot_stride % 8 || c->v_head_stride % 8 ||
        q_token % qn || q_head % qn || out_token % on || out_head % on)
        return Q4K_ERR_MISALIGNED;
    int sms = 0;
    st = check_device(&sms);
    if (st != Q4K_OK || !some) return st;

    attn::RowsLaunch l{};
    attn::Args &p = l.args;
    p.q = a->q, p.k = c->k, p.v = c->v, p.out = a->out, p.lse = a->lse;
    p.q_token = q_token, p.q_head = q_head, p.out_token = out_token, p.out_head = out_head;
    p.k_page = c->k_page_stride, p.k_slot = c->k_slot_stride, p.k_head = c->k_head_stride;
    p.v_page = c->v_page_stride, p.v_slot = c->v_slot_stride, p.v_head = c->v_head_stride;
    p.table_stride = c->page_table_stride, p.page_size = static_cast<int>(c->page_size);
    p.page_shift = -1;
    if ((c->page_size & (c->page_size - 1)) == 0)
        for (p.page_shift = 0; (int64_t{1} << p.page_shift) < c->page_size;) ++p.page_shift;
    p.page_table = c->page_table, p.seq_start = c->seq_start, p.kv_len = c->kv_len;
    p.prefix_len = a->prefix_len, p.kv_start = a->kv_start, p.slopes = a->slopes;
    // positions are 32-bit in the kernels, with room above them
    const int64_t most = 0x3FFFFFFF;
    const int64_t per = c->pages > 0 ? c->max_pages : 0;
    p.capacity = static_cast<int>(per > most / c->page_size ? most : per * c->page_size);
    // a window past every position is none
    p.window = a->window > most ? 0 : static_cast<int>(a->window), p.scale = a->scale;
    // beyond 1e30 a cap is none that fp32 scores could tell, below 1e-30 all scores are alike;
    // the quotient and products with it stay normal numbers
    p.softcap = a->softcap > 0.0f ? std::min(std::max(a->softcap, 1e-30f), 1e30f) : 0.0f;
    p.pages = static_cast<int>(c->pages), p.batch = static_cast<int>(c->batch);
    p.tokens = static_cast<int>(c->tokens), p.heads = static_cast<int>(a->q_heads);
    p.kv_heads = static_cast<int>(c->heads), p.group = static_cast<int>(a->q_heads / c->heads);
    p.dim = static_cast<int>(c->dim), p.q_type = a->q_type, p.out_type = a->out_type, p.causal = a->causal;
    p.wait_ns = a->wait_limit_us ? 1000ull * a->wait_limit_us : 2000000000ull;
    p.stall = (a->flags & Q4K_FLAG_TEST_STALL) != 0;
    p.pdl = (a->flags & Q4K_FLAG_PDL) != 0;
    if (cudaGetDevice(&l.device) != cudaSuccess || l.device < 0 || l.device >= attn::kDevices ||
        error_word(l.device, &p.error) != cudaSuccess)
        return Q4K_ERR_CUDA;
    l.sms = sms;
    l.stream = static_cast<cudaStream_t>(stream);
    // 16-bit calls form cap tanh(s / cap) as cap (1 - 2 / (exp + 1)), off by 2^-22 of the cap:
    // at 256 an eighth of what rounding a weight to fp16 may cost.  Larger caps take the
    // kernels of fp32 calls, whose tanh is good to a few ulp of itself.
    l.parts_many = a->q_type != c->type || a->out_type == Q4K_F32 || p.softcap > 256.0f;
    // The tcgen05 kernel takes q of the cache's type, a 16-bit out and pages that split into
    // boxes of 16 slots or more.  Its TMA boxes also ask for positive strides and
    // groups of 256 heads at most, its maxima for a scale that is not negative.
    auto stride_ok = [](int64_t s) { return s > 0 && s < (int64_t{1} << 39); };
    const bool boxes = c->page_size % 16 == 0 && stride_ok(c->k_slot_stride) && stride_ok(c->v_slot_stride) &&
                       (c->heads == 1 || (stride_ok(c->k_head_stride) && stride_ok(c->v_head_stride))) &&
                       (c->pages == 1 || (stride_ok(c->k_page_stride) && stride_ok(c->v_page_stride)));
    l.boxes = boxes && p.capacity > 0;
    const bool queries = p.group <= attn::kChunkRows && a->scale >= 0.0f &&
                         (c->tokens == 1 || stride_ok(q_token)) && (a->q_heads == 1 || stride_ok(q_head));
    const int (*room)[attn::kMaxCluster + 1];
    if (attn::room_of(l.device, &room) != cudaSuccess) return Q4K_ERR_CUDA;
    const int parts = !l.parts_many ? 1 : c->type == Q4K_F16 ? 2 : 3;
    l.choice = attn::choose(p, *room, sms, parts, !l.parts_many && c->dim <= 128 && l.boxes && queries,
                            static_cast<int>(a->flags >> 8 & 7));
    if (!l.choice.chunk && !l.choice.rows) return Q4K_ERR_INVALID_ARG;
    cudaError_t e;
    if (l.choice.chunk) {
        const attn::ChunkLaunch ch{p, l.device, sms, l.stream};
        e = c->type == Q4K_F16 ? attn::launch_chunk_f16(ch) : attn::launch_chunk_bf16(ch);
    } else {
        auto rows = c->type == Q4K_F16 ? (p.docs() ? attn::launch_rows_docs_f16 : attn::launch_rows_f16)
                                       : (p.docs() ? attn::launch_rows_docs_bf16 : attn::launch_rows_bf16);
        e = rows(l);
    }
    return e == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA;
}

}  // namespace q4k
