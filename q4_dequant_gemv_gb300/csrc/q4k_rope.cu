// q4k_rope.cu -- rotary positions (q4k_rope_table, q4k_rope) and the append of
// new keys and values to a paged cache with the rotation on the way
// (q4k_kv_append).
//
// A pair (a, b) of a head turns by its token's angle: a' = a c - b s,
// b' = a s + b c, with c, s from a table made once in fp64.  Three flops per
// value against 4 to 8 bytes moved: bound by memory (or, for a few tokens, by
// the chain of dependent index loads).
//
// One CTA per token.  A thread owns one unit of a head (8 pairs, or 16 copied
// elements) and walks the heads, so a table row is loaded once per thread and
// not once per head; all data moves in 16-byte accesses where rows are 16-byte
// aligned and the sizes are multiples of 16, element by element otherwise.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/q4k.h"
#include "q4k_attn.cuh"
#include "q4k_internal.h"

namespace q4k {

__device__ unsigned int g_rope_error = 0;   // bit 2: an index outside its buffer

unsigned int read_rope_error()
{
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    return v;
}

bool clear_rope_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_rope_error, &z, sizeof(z)) == cudaSuccess;
}

namespace rope {

constexpr int kMaxRot = 512;
constexpr int kThreads = 256;

struct Freqs {
    double f[kMaxRot / 2];
    double magnitude;
};

__global__ void __launch_bounds__(kThreads) table_kernel(float *table, int64_t rows, int half, const Freqs fr)
{
    const int64_t n = rows * half;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t p = i / half;
        const int j = static_cast<int>(i - p * half);
        double s, c;
        sincos(static_cast<double>(p) * fr.f[j], &s, &c);
        table[p * 2 * half + j] = static_cast<float>(c * fr.magnitude);
        table[p * 2 * half + half + j] = static_cast<float>(s * fr.magnitude);
    }
}

// A [heads][dim] row per token, source and destination.
struct Rows {
    const void *x;
    void *y;
    int64_t xt, xh, yt, yh;   // strides in elements (yt unused for the cache)
    int heads, xtype, ytype;
};

__device__ __forceinline__ void load8(const void *p, int type, int64_t i, float (&f)[8])
{
    if (type == Q4K_F32) {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = s[0], b = s[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = attn::unpack2(w[j], type);
            f[2 * j] = t.x, f[2 * j + 1] = t.y;
        }
    }
}

__device__ __forceinline__ void store8(void *p, int type, int64_t i, const float (&f)[8])
{
    if (type == Q4K_F32) {
        float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        d[0] = make_float4(f[0], f[1], f[2], f[3]);
        d[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
            make_uint4(attn::pack2(f[0], f[1], type), attn::pack2(f[2], f[3], type), attn::pack2(f[4], f[5], type),
                       attn::pack2(f[6], f[7], type));
    }
}

__device__ __forceinline__ float load1(const void *p, int type, int64_t i)
{
    if (type == Q4K_F32) return static_cast<const float *>(p)[i];
    if (type == Q4K_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ void store1(void *p, int type, int64_t i, float v)
{
    if (type == Q4K_F32) static_cast<float *>(p)[i] = v;
    else if (type == Q4K_F16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// One token's heads of one tensor, by the calling CTA.  x and y already point
// at the token's row.  rot = 0 copies.  Wide path: units of 16 elements, unit u
// < rot/16 turns pairs 8u..8u+7, the others copy elements 16u..16u+15.
template <bool WIDE>
__device__ __forceinline__ void turn_rows(const Rows &r, int64_t x0, int64_t y0, int dim, int rot, int inter,
                                          const float *trow)
{
    const int half = rot >> 1;
    if (WIDE) {
        const int units = (dim + 15) >> 4, turned = rot >> 4;
        const int lanes = kThreads / units;   // heads in flight (units <= 64 on this path)
        const int u = threadIdx.x % units;
        int h = threadIdx.x / units;
        if (h >= lanes) return;
        if (u < turned) {
            float c[8], s[8];
            load8(trow, Q4K_F32, 8 * u, c);
            load8(trow, Q4K_F32, half + 8 * u, s);
            const int ia = inter ? 16 * u : 8 * u, ib = inter ? ia + 8 : ia + half;
            for (; h < r.heads; h += lanes) {
                float a[8], b[8], p[8], q[8];
                load8(r.x, r.xtype, x0 + h * r.xh + ia, a);
                load8(r.x, r.xtype, x0 + h * r.xh + ib, b);
                if (inter) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[2 * j] = a[2 * j] * c[j] - a[2 * j + 1] * s[j];
                        p[2 * j + 1] = a[2 * j] * s[j] + a[2 * j + 1] * c[j];
                        q[2 * j] = b[2 * j] * c[4 + j] - b[2 * j + 1] * s[4 + j];
                        q[2 * j + 1] = b[2 * j] * s[4 + j] + b[2 * j + 1] * c[4 + j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        p[j] = a[j] * c[j] - b[j] * s[j];
                        q[j] = a[j] * s[j] + b[j] * c[j];
                    }
                }
                store8(r.y, r.ytype, y0 + h * r.yh + ia, p);
                store8(r.y, r.ytype, y0 + h * r.yh + ib, q);
            }
        } else {
            const bool two = 16 * u + 16 <= dim;
            for (; h < r.heads; h += lanes) {
                float a[8], b[8];
                load8(r.x, r.xtype, x0 + h * r.xh + 16 * u, a);
                if (two) load8(r.x, r.xtype, x0 + h * r.xh + 16 * u + 8, b);
                store8(r.y, r.ytype, y0 + h * r.yh + 16 * u, a);
                if (two) store8(r.y, r.ytype, y0 + h * r.yh + 16 * u + 8, b);
            }
        }
    } else {
        const int per = half + (dim - rot);   // pairs, then copied elements
        for (int64_t i = threadIdx.x; i < static_cast<int64_t>(per) * r.heads; i += kThreads) {
            const int h = static_cast<int>(i / per), u = static_cast<int>(i - static_cast<int64_t>(h) * per);
            const int64_t x = x0 + h * r.xh, y = y0 + h * r.yh;
            if (u < half) {
                const int ia = inter ? 2 * u : u, ib = inter ? ia + 1 : u + half;
                const float c = trow[u], s = trow[half + u];
                const float a = load1(r.x, r.xtype, x + ia), b = load1(r.x, r.xtype, x + ib);
                store1(r.y, r.ytype, y + ia, a * c - b * s);
                store1(r.y, r.ytype, y + ib, a * s + b * c);
            } else {
                const int d = rot + (u - half);
                store1(r.y, r.ytype, y + d, load1(r.x, r.xtype, x + d));
            }
        }
    }
}

template <bool WIDE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Rows r, const int32_t *pos, const float *table,
                                                        int64_t table_rows, int dim, int rot, int inter)
{
    const int64_t t = blockIdx.x;
    const float *trow = nullptr;
    if (rot) {
        const int p = pos[t];
        if (p < 0 || p >= table_rows) {
            if (threadIdx.x == 0) atomicOr(&g_rope_error, 4u);
            return;
        }
        trow = table + static_cast<int64_t>(p) * rot;
    }
    turn_rows<WIDE>(r, t * r.xt, t * r.yt, dim, rot, inter, trow);
}

struct AppendArgs {
    Rows q, k, v;
    int64_t k_page, k_slot, v_page, v_slot;
    int64_t pages, page_size, table_stride, max_pages, table_rows;
    const int32_t *page_table, *seq_start, *kv_len, *pos;
    const float *table;
    int batch, tokens, dim, rot, inter;
};

// blockIdx.x = token.  The CTA finds its sequence (one comparison per thread and
// 256 sequences), then its slot, and writes q_out, the key and the value.
template <bool WIDE>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a)
{
    __shared__ int s_seq, s_first, s_end;
    const int t = blockIdx.x;
    if (threadIdx.x == 0) s_seq = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
        const int lo = a.seq_start[b], hi = a.seq_start[b + 1];
        if (t >= lo && t < hi) s_seq = b, s_first = lo, s_end = hi;
    }
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    // a token of a sequence outside the call's rows, or before position 0
    const int64_t p = static_cast<int64_t>(a.kv_len[b]) - (s_end - s_first) + (t - s_first);
    bool ok = s_first >= 0 && s_end <= a.tokens && p >= 0 && p / a.page_size < a.max_pages;
    const int64_t row = a.rot ? (a.pos ? static_cast<int64_t>(a.pos[t]) : p) : 0;
    if (a.rot && (row < 0 || row >= a.table_rows)) ok = false;
    int64_t page = 0;
    if (ok) {
        page = a.page_table[b * a.table_stride + p / a.page_size];
        ok = page >= 0 && page < a.pages;
    }
    if (!ok) {
        if (threadIdx.x == 0) atomicOr(&g_rope_error, 4u);
        return;
    }
    const int64_t slot = p % a.page_size;
    const float *trow = a.rot ? a.table + row * a.rot : nullptr;
    turn_rows<WIDE>(a.k, t * a.k.xt, page * a.k_page + slot * a.k_slot, a.dim, a.rot, a.inter, trow);
    turn_rows<WIDE>(a.v, t * a.v.xt, page * a.v_page + slot * a.v_slot, a.dim, 0, 0, nullptr);
    if (a.q.x) turn_rows<WIDE>(a.q, t * a.q.xt, t * a.q.yt, a.dim, a.rot, a.inter, trow);
}

static bool good_type(int t) { return t == Q4K_F32 || t == Q4K_F16 || t == Q4K_BF16; }
static int size_of(int t) { return t == Q4K_F32 ? 4 : 2; }
static bool off(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Whether every head row of a tensor starts on a 16-byte boundary.
static bool wide_rows(const void *p, int type, int64_t token_stride, int64_t head_stride)
{
    const int64_t per = 16 / size_of(type);
    return !off(p, 16) && token_stride % per == 0 && head_stride % per == 0;
}

}  // namespace rope

q4k_status rope_table_impl(float *table, int64_t rows, int64_t rot, const q4k_rope_scaling *s, void *stream)
{
    if (!s || rows < 0 || rot < 2 || rot > rope::kMaxRot || rot % 2 || (rows > 0 && !table)) return Q4K_ERR_INVALID_ARG;
    if (!(s->base > 0) || !(s->factor > 0) || !std::isfinite(s->base) || !std::isfinite(s->factor) ||
        !std::isfinite(s->magnitude) || s->scaling < Q4K_ROPE_PLAIN || s->scaling > Q4K_ROPE_BANDS)
        return Q4K_ERR_INVALID_ARG;
    if (s->scaling >= Q4K_ROPE_RAMP && (!(s->orig_len > 0) || !(s->low > 0) || !(s->high > s->low) ||
                                        !std::isfinite(s->orig_len) || !std::isfinite(s->high)))
        return Q4K_ERR_INVALID_ARG;
    if (s->scaling == Q4K_ROPE_BASE && rot == 2) return Q4K_ERR_INVALID_ARG;
    if (s->scaling == Q4K_ROPE_RAMP && s->base == 1.0) return Q4K_ERR_INVALID_ARG;
    if (rope::off(table, 4)) return Q4K_ERR_MISALIGNED;
    q4k_status st = check_device(nullptr);
    if (st != Q4K_OK || rows == 0) return st;
    const double two_pi = 6.283185307179586476925286766559;
    rope::Freqs fr;
    fr.magnitude = s->magnitude;
    const double n = static_cast<double>(rot);
    const double base = s->scaling == Q4K_ROPE_BASE ? s->base * std::pow(s->factor, n / (n - 2)) : s->base;
    // RAMP: the pair index that turns r times over orig_len positions
    auto pair_of = [&](double r) { return n * std::log(s->orig_len / (r * two_pi)) / (2 * std::log(base)); };
    double first = 0, last = 0;
    if (s->scaling == Q4K_ROPE_RAMP) {
        first = std::fmax(std::floor(pair_of(s->high)), 0.0);
        last = std::fmin(std::ceil(pair_of(s->low)), n - 1);
        if (!(last > first)) last = first + 0.001;   // a step
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / n);
        double g = f;
        if (s->scaling == Q4K_ROPE_LINEAR) g = f / s->factor;
        if (s->scaling == Q4K_ROPE_RAMP) {
            const double r = std::fmin(std::fmax((i - first) / (last - first), 0.0), 1.0);
            g = f / s->factor * r + f * (1 - r);
        }
        if (s->scaling == Q4K_ROPE_BANDS) {
            const double turns = s->orig_len * f / two_pi;   // orig_len / wavelength
            if (turns < s->low) g = f / s->factor;
            else if (turns <= s->high) {
                const double m = (turns - s->low) / (s->high - s->low);
                g = (1 - m) * f / s->factor + m * f;
            }
        }
        fr.f[i] = g;
    }
    const int64_t n_all = rows * (rot / 2);
    const int64_t blocks = (n_all + rope::kThreads - 1) / rope::kThreads;
    rope::table_kernel<<<static_cast<unsigned>(blocks < 16384 ? blocks : 16384), rope::kThreads, 0,
                         static_cast<cudaStream_t>(stream)>>>(table, rows, static_cast<int>(rot / 2), fr);
    return cudaGetLastError() == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA;
}

q4k_status rope_impl(const q4k_rope_args *a, void *stream)
{
    using namespace rope;
    if (!a || a->tokens < 0 || a->tokens > 0x7FFFFFFF || a->heads < 1 || a->heads > 65536 || a->dim < 1 ||
        a->dim > 65536 || a->rot < 0 || a->rot % 2 || a->rot > a->dim || a->rot > kMaxRot || a->table_rows < 0 ||
        !good_type(a->x_type) || !good_type(a->y_type) || (a->interleaved & ~1))
        return Q4K_ERR_INVALID_ARG;
    if (a->tokens > 0 && (!a->x || !a->y || (a->rot && (!a->pos || !a->table)))) return Q4K_ERR_INVALID_ARG;
    if (off(a->x, size_of(a->x_type)) || off(a->y, size_of(a->y_type)) || off(a->pos, 4) || off(a->table, 4))
        return Q4K_ERR_MISALIGNED;
    q4k_status st = check_device(nullptr);
    if (st != Q4K_OK || a->tokens == 0) return st;
    const Rows r{a->x, a->y, a->x_token_stride, a->x_head_stride, a->y_token_stride, a->y_head_stride,
                 static_cast<int>(a->heads), a->x_type, a->y_type};
    const bool wide = a->dim % 8 == 0 && a->dim <= 1024 && a->rot % 16 == 0 && !off(a->table, 16) &&
                      wide_rows(a->x, a->x_type, r.xt, r.xh) && wide_rows(a->y, a->y_type, r.yt, r.yh);
    auto kern = wide ? rope_kernel<true> : rope_kernel<false>;
    kern<<<static_cast<unsigned>(a->tokens), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        r, a->pos, a->table, a->table_rows, static_cast<int>(a->dim), static_cast<int>(a->rot), a->interleaved);
    return cudaGetLastError() == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA;
}

q4k_status check_cache(const q4k_paged_cache *c)
{
    using namespace rope;
    if (!c || c->batch < 0 || c->batch > 0x7FFFFFF || c->tokens < 0 || c->tokens > 0x7FFFFFFF || c->pages < 0 ||
        c->pages > 0x7FFFFFFF || c->page_size < 1 || c->page_size > 0x7FFFFFFF || c->heads < 1 || c->heads > 65536 ||
        c->dim < 1 || c->dim > 65536 || c->max_pages < 0 || c->page_table_stride < 0 ||
        (c->type != Q4K_F16 && c->type != Q4K_BF16))
        return Q4K_ERR_INVALID_ARG;
    if (c->tokens > 0 && c->batch > 0 && (!c->k || !c->v || !c->page_table || !c->seq_start || !c->kv_len))
        return Q4K_ERR_INVALID_ARG;
    if (off(c->k, 2) || off(c->v, 2) || off(c->page_table, 4) || off(c->seq_start, 4) || off(c->kv_len, 4))
        return Q4K_ERR_MISALIGNED;
    return Q4K_OK;
}

q4k_status kv_append_impl(const q4k_paged_cache *c, const q4k_append_args *a, void *stream)
{
    using namespace rope;
    q4k_status st = check_cache(c);
    if (st == Q4K_ERR_INVALID_ARG || !a) return Q4K_ERR_INVALID_ARG;
    const bool some = c->tokens > 0 && c->batch > 0;
    if (a->rot < 0 || a->rot % 2 || a->rot > c->dim || a->rot > kMaxRot || a->table_rows < 0 ||
        !good_type(a->kv_type) || (a->interleaved & ~1) || (a->q == nullptr) != (a->q_out == nullptr))
        return Q4K_ERR_INVALID_ARG;
    if (a->q && (a->q_heads < 1 || a->q_heads > 65536 || !good_type(a->q_type) || !good_type(a->q_out_type)))
        return Q4K_ERR_INVALID_ARG;
    if (some && (!a->k || !a->v || (a->rot && !a->table))) return Q4K_ERR_INVALID_ARG;
    if (st != Q4K_OK) return st;
    if (off(a->k, size_of(a->kv_type)) || off(a->v, size_of(a->kv_type)) || off(a->pos, 4) || off(a->table, 4) ||
        (a->q && (off(a->q, size_of(a->q_type)) || off(a->q_out, size_of(a->q_out_type)))))
        return Q4K_ERR_MISALIGNED;
    st = check_device(nullptr);
    if (st != Q4K_OK || !some) return st;
    AppendArgs p{};
    const int heads = static_cast<int>(c->heads);
    p.k = Rows{a->k, c->k, a->k_token_stride, a->k_head_stride, 0, c->k_head_stride, heads, a->kv_type, c->type};
    p.v = Rows{a->v, c->v, a->v_token_stride, a->v_head_stride, 0, c->v_head_stride, heads, a->kv_type, c->type};
    if (a->q)
        p.q = Rows{a->q, a->q_out, a->q_token_stride, a->q_head_stride, a->q_out_token_stride, a->q_out_head_stride,
                   static_cast<int>(a->q_heads), a->q_type, a->q_out_type};
    p.k_page = c->k_page_stride, p.k_slot = c->k_slot_stride, p.v_page = c->v_page_stride, p.v_slot = c->v_slot_stride;
    p.pages = c->pages, p.page_size = c->page_size, p.table_stride = c->page_table_stride, p.max_pages = c->max_pages;
    p.page_table = c->page_table, p.seq_start = c->seq_start, p.kv_len = c->kv_len, p.pos = a->pos;
    p.table = a->table, p.table_rows = a->table_rows;
    p.batch = static_cast<int>(c->batch), p.tokens = static_cast<int>(c->tokens), p.dim = static_cast<int>(c->dim);
    p.rot = static_cast<int>(a->rot), p.inter = a->interleaved;
    bool wide = c->dim % 8 == 0 && c->dim <= 1024 && a->rot % 16 == 0 && !off(a->table, 16) &&
                wide_rows(a->k, a->kv_type, p.k.xt, p.k.xh) && wide_rows(a->v, a->kv_type, p.v.xt, p.v.xh) &&
                wide_rows(c->k, c->type, p.k_page, p.k_slot) && wide_rows(c->v, c->type, p.v_page, p.v_slot) &&
                p.k.yh % 8 == 0 && p.v.yh % 8 == 0;
    if (a->q)
        wide = wide && wide_rows(a->q, a->q_type, p.q.xt, p.q.xh) && wide_rows(a->q_out, a->q_out_type, p.q.yt, p.q.yh);
    auto kern = wide ? append_kernel<true> : append_kernel<false>;
    kern<<<static_cast<unsigned>(c->tokens), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA;
}

}  // namespace q4k
