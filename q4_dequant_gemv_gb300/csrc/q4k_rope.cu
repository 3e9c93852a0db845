// q4k_rope.cu -- rotary positions (q4k_rope_table, q4k_rope) and the append of
// new keys and values to a paged cache with the rotation on the way
// (q4k_kv_append).
//
// A pair (a, b) of a head turns by its token's angle: a' = a c - b s,
// b' = a s + b c, with c, s from a table made once in fp64.  Three flops per
// value against 4 to 8 bytes moved: bound by memory (or, for a few tokens, by
// the chain of dependent index loads).
//
// A token's heads (of q, k and v alike) are cut into units of 8 pairs or 16
// copied elements, a unit per thread, in as many warps as that takes; small
// tokens share a CTA.  The data's loads are issued before the chain of index
// loads (sequence, length, page and table row) that the stores wait for, so a
// call needs three dependent trips to memory; warps find their sequence by
// themselves, and nothing synchronises a CTA.  All data moves in 16-byte
// accesses where rows are 16-byte aligned and the sizes are multiples of 16,
// element by element otherwise.

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
constexpr int kThreads = 512;

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

// Heads of one tensor: source and destination of a token.
struct Part {
    const void *x;
    void *y;
    int64_t xt, xh, yt, yh;   // strides in elements (yt: of a token, or unused for the cache)
    int heads, xtype, ytype;
    int rot;                  // turned elements of a head (0: copied)
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

struct TokenArgs {
    Part part[3];             // rope: one; append: keys, values, queries (heads = 0: absent)
    int64_t k_page, k_slot, v_page, v_slot;
    int64_t pages, page_size, table_stride, max_pages, table_rows;
    const int32_t *page_table, *seq_start, *kv_len, *pos;
    const float *table;
    int batch, tokens, dim, rot, inter;
    int units, items;         // per head, per token
    int warps;                // of a token
};

// The last sequence that starts at or before token t (-1: none), by a whole warp
// in steps of 32-way division.
__device__ __forceinline__ int find_sequence(const int32_t *start, int batch, int t)
{
    int lo = 0, n = batch;    // the answer is lo - 1 or one of [lo, lo + n)
    const int lane = threadIdx.x & 31;
    while (true) {
        const int step = (n + 31) / 32, i = lane * step;
        const bool below = i < n && start[lo + i] <= t;
        const int k = __popc(__ballot_sync(0xffffffffu, below));
        if (k == 0) return lo - 1;
        const int skip = (k - 1) * step;
        lo += skip;
        if (step == 1) return lo;
        n = min(step, n - skip);
    }
}

struct Unit {
    int part, head, ia, ib;   // tensor, head, first elements of its two halves
    bool turned, two;         // two: the second half exists
};

__device__ __forceinline__ Unit unit_of(const TokenArgs &a, int i)
{
    Unit u;
    int h = i / a.units;
    const int j = i - h * a.units;
    u.part = 0;
    while (h >= a.part[u.part].heads) h -= a.part[u.part].heads, ++u.part;
    u.head = h;
    const int rot = a.part[u.part].rot;
    u.turned = 16 * j < rot;
    u.ia = u.turned && !a.inter ? 8 * j : 16 * j;
    u.ib = u.turned && !a.inter ? u.ia + (rot >> 1) : u.ia + 8;
    u.two = u.ib < a.dim;
    return u;
}

__device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], const float (&c)[8], const float (&s)[8], int inter)
{
    float p[8], q[8];
    if (inter) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[2 * j] = x[2 * j] * c[j] - x[2 * j + 1] * s[j];
            p[2 * j + 1] = x[2 * j] * s[j] + x[2 * j + 1] * c[j];
            q[2 * j] = y[2 * j] * c[4 + j] - y[2 * j + 1] * s[4 + j];
            q[2 * j + 1] = y[2 * j] * s[4 + j] + y[2 * j + 1] * c[4 + j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = x[j] * c[j] - y[j] * s[j];
            q[j] = x[j] * s[j] + y[j] * c[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = p[j], y[j] = q[j];
}

template <bool WIDE, bool APPEND>
__global__ void __launch_bounds__(kThreads) token_kernel(const TokenArgs a)
{
    const int w = threadIdx.x >> 5;
    const int per = static_cast<int>(blockDim.x >> 5) / a.warps;   // tokens of a CTA
    const int64_t t = static_cast<int64_t>(blockIdx.x) * per + w / a.warps;
    if (t >= a.tokens) return;
    const int first = (w % a.warps) * 32 + (threadIdx.x & 31), step = a.warps * 32;

    float x[8], y[8];
    Unit u{};
    if (WIDE && first < a.items) {
        u = unit_of(a, first);
        const Part &p = a.part[u.part];
        load8(p.x, p.xtype, t * p.xt + u.head * p.xh + u.ia, x);
        if (u.two) load8(p.x, p.xtype, t * p.xt + u.head * p.xh + u.ib, y);
    }

    // ---- where the token goes and which table row turns it
    int64_t row = 0, at_k = 0, at_v = 0;
    bool ok = true;
    if (APPEND) {
        const int b = find_sequence(a.seq_start, a.batch, static_cast<int>(t));
        if (b < 0) return;
        const int s0 = a.seq_start[b], s1 = a.seq_start[b + 1];
        if (t >= s1) return;   // a token of no sequence
        const int64_t p = static_cast<int64_t>(a.kv_len[b]) - s1 + t;
        row = a.rot ? (a.pos ? static_cast<int64_t>(a.pos[t]) : p) : 0;
        ok = s0 >= 0 && s1 <= a.tokens && p >= 0 && p / a.page_size < a.max_pages && (!a.rot || (row >= 0 && row < a.table_rows));
        if (ok) {
            const int64_t e = p / a.page_size, slot = p - e * a.page_size;
            const int64_t page = a.page_table[b * a.table_stride + e];
            ok = page >= 0 && page < a.pages;
            at_k = page * a.k_page + slot * a.k_slot, at_v = page * a.v_page + slot * a.v_slot;
        }
    } else if (a.rot) {
        row = a.pos[t];
        ok = row >= 0 && row < a.table_rows;
    }
    if (!ok) {
        if (first == 0) atomicOr(&g_rope_error, 4u);
        return;
    }
    const float *trow = a.table + row * a.rot;
    auto dest = [&](int part) { return APPEND ? (part == 0 ? at_k : part == 1 ? at_v : t * a.part[2].yt) : t * a.part[0].yt; };

    if (WIDE) {
        for (int i = first; i < a.items; i += step) {
            if (i != first) {
                u = unit_of(a, i);
                const Part &p = a.part[u.part];
                load8(p.x, p.xtype, t * p.xt + u.head * p.xh + u.ia, x);
                if (u.two) load8(p.x, p.xtype, t * p.xt + u.head * p.xh + u.ib, y);
            }
            const Part &p = a.part[u.part];
            if (u.turned) {
                const int j = a.inter ? u.ia >> 1 : u.ia;   // first pair
                float c[8], s[8];
                load8(trow, Q4K_F32, j, c);
                load8(trow, Q4K_F32, (a.rot >> 1) + j, s);
                turn(x, y, c, s, a.inter);
            }
            const int64_t o = dest(u.part) + u.head * p.yh;
            store8(p.y, p.ytype, o + u.ia, x);
            if (u.two) store8(p.y, p.ytype, o + u.ib, y);
        }
    } else {
        // element by element: a head is its pairs, then its copied elements
        for (int q = 0; q < (APPEND ? 3 : 1); ++q) {
            const Part &p = a.part[q];
            const int half = p.rot >> 1, each = half + (a.dim - p.rot);
            for (int64_t i = first; i < static_cast<int64_t>(each) * p.heads; i += step) {
                const int h = static_cast<int>(i / each), j = static_cast<int>(i - static_cast<int64_t>(h) * each);
                const int64_t from = t * p.xt + h * p.xh, to = dest(q) + h * p.yh;
                if (j < half) {
                    const int ia = a.inter ? 2 * j : j, ib = a.inter ? ia + 1 : j + half;
                    const float c = trow[j], s = trow[half + j];
                    const float v = load1(p.x, p.xtype, from + ia), z = load1(p.x, p.xtype, from + ib);
                    store1(p.y, p.ytype, to + ia, v * c - z * s);
                    store1(p.y, p.ytype, to + ib, v * s + z * c);
                } else {
                    const int d = p.rot + (j - half);
                    store1(p.y, p.ytype, to + d, load1(p.x, p.xtype, from + d));
                }
            }
        }
    }
}

// Warps per token and tokens per CTA, then the launch.
template <bool APPEND>
static q4k_status launch_tokens(TokenArgs &a, bool wide, void *stream)
{
    int64_t heads = 0;
    for (const Part &p : a.part) heads += p.heads;
    a.units = (a.dim + 15) / 16;
    const int64_t items = heads * (wide ? a.units : a.dim);
    if (items > 0x7FFFFFFF) return Q4K_ERR_INVALID_ARG;
    a.items = static_cast<int>(items);
    const int64_t need = (items + 31) / 32, rounds = (need + kThreads / 32 - 1) / (kThreads / 32);
    a.warps = static_cast<int>((need + rounds - 1) / rounds);
    const int per = a.warps >= 4 ? 1 : 4 / a.warps;   // tokens of a CTA: four warps or more
    const int64_t grid = (static_cast<int64_t>(a.tokens) + per - 1) / per;
    auto kern = wide ? token_kernel<true, APPEND> : token_kernel<false, APPEND>;
    kern<<<static_cast<unsigned>(grid), a.warps * per * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA;
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
    TokenArgs p{};
    p.part[0] = Part{a->x, a->y, a->x_token_stride, a->x_head_stride, a->y_token_stride, a->y_head_stride,
                     static_cast<int>(a->heads), a->x_type, a->y_type, static_cast<int>(a->rot)};
    p.pos = a->pos, p.table = a->table, p.table_rows = a->table_rows;
    p.tokens = static_cast<int>(a->tokens), p.dim = static_cast<int>(a->dim), p.rot = static_cast<int>(a->rot);
    p.inter = a->interleaved;
    const Part &r = p.part[0];
    const bool wide = a->dim % 8 == 0 && a->rot % 16 == 0 && !off(a->table, 16) &&
                      wide_rows(a->x, a->x_type, r.xt, r.xh) && wide_rows(a->y, a->y_type, r.yt, r.yh);
    return launch_tokens<false>(p, wide, stream);
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
    TokenArgs p{};
    const int heads = static_cast<int>(c->heads), rot = static_cast<int>(a->rot);
    p.part[0] = Part{a->k, c->k, a->k_token_stride, a->k_head_stride, 0, c->k_head_stride, heads, a->kv_type, c->type, rot};
    p.part[1] = Part{a->v, c->v, a->v_token_stride, a->v_head_stride, 0, c->v_head_stride, heads, a->kv_type, c->type, 0};
    if (a->q)
        p.part[2] = Part{a->q, a->q_out, a->q_token_stride, a->q_head_stride, a->q_out_token_stride,
                         a->q_out_head_stride, static_cast<int>(a->q_heads), a->q_type, a->q_out_type, rot};
    p.k_page = c->k_page_stride, p.k_slot = c->k_slot_stride, p.v_page = c->v_page_stride, p.v_slot = c->v_slot_stride;
    p.pages = c->pages, p.page_size = c->page_size, p.table_stride = c->page_table_stride, p.max_pages = c->max_pages;
    p.page_table = c->page_table, p.seq_start = c->seq_start, p.kv_len = c->kv_len, p.pos = a->pos;
    p.table = a->table, p.table_rows = a->table_rows;
    p.batch = static_cast<int>(c->batch), p.tokens = static_cast<int>(c->tokens), p.dim = static_cast<int>(c->dim);
    p.rot = rot, p.inter = a->interleaved;
    const Part &k = p.part[0], &v = p.part[1], &q = p.part[2];
    bool wide = c->dim % 8 == 0 && rot % 16 == 0 && !off(a->table, 16) && wide_rows(a->k, a->kv_type, k.xt, k.xh) &&
                wide_rows(a->v, a->kv_type, v.xt, v.xh) && wide_rows(c->k, c->type, p.k_page, p.k_slot) &&
                wide_rows(c->v, c->type, p.v_page, p.v_slot) && k.yh % 8 == 0 && v.yh % 8 == 0;
    if (a->q) wide = wide && wide_rows(a->q, a->q_type, q.xt, q.xh) && wide_rows(a->q_out, a->q_out_type, q.yt, q.yh);
    return launch_tokens<true>(p, wide, stream);
}

}  // namespace q4k
