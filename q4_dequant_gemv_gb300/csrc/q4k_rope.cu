// q4k_rope.cu -- rotary positions (q4k_rope_table, q4k_rope) and the append of
// new keys and values to a paged cache with the rotation on the way
// (q4k_kv_append).
//
// A pair (a, b) of a head turns by its token's angle: a' = a c - b s,
// b' = a s + b c, with c, s from a table made once in fp64.  Three flops per
// value against 4 to 8 bytes moved: bound by memory (or, for a few tokens, by
// the chain of dependent index loads).
//
// A token's heads (of q, k and v alike) are cut into units of 4 pairs or 8
// copied elements, a unit per thread, in as many warps as that takes; small
// tokens share a CTA.  With many tokens a thread takes the same unit of four of
// them: all their data is on its way before the chain of index loads (sequence,
// length, page, table row) begins, and four lanes of each warp follow the four
// chains at once.  Nothing synchronises a CTA.  Data moves in accesses of four
// elements where rows are 16-byte aligned and the sizes are multiples of 8,
// element by element otherwise.
//
// Measured: 4097 tokens of 32 bf16 heads, half of each turned, 14.1 us (68 MB,
// 4.8 TB/s from memory and L2; a plain copy of as much 11.7); append of 2048 fp32
// tokens of 28 + 8 heads 14.9 us, of three fp16 prompts of 2500 15.0; one token
// 1.9, sixteen with their page lookups 2.9.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/q4k.h"
#include "ptx.cuh"
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
constexpr int kThreads = 128;   // of a CTA at most
constexpr int kTok = 4;         // tokens of a thread in large calls

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

template <int TYPE>
__device__ __forceinline__ void convert4(const uint2 &r, float (&f)[4])
{
    const float2 a = attn::unpack2(r.x, TYPE), b = attn::unpack2(r.y, TYPE);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}

template <int TYPE>
__device__ __forceinline__ void convert4(const uint4 &r, float (&f)[4])
{
    if constexpr (TYPE == Q4K_F32) {
        f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y), f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
    } else {
        const float2 a = attn::unpack2(r.x, TYPE), b = attn::unpack2(r.y, TYPE);
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    }
}

template <int TYPE>
__device__ __forceinline__ void store4(uint8_t *p, const float (&f)[4])
{
    if constexpr (TYPE == Q4K_F32) *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(attn::pack2(f[0], f[1], TYPE), attn::pack2(f[2], f[3], TYPE));
}

// TOK tokens' unit: converted, turned by their c and s (kind 1: halves apart,
// kind 2: neighbours, 0: copied) and stored where `to` is not null.
template <int XT, int YT, int TOK, class Raw>
__device__ __forceinline__ void finish(const Raw *ra, const Raw *rb, const float4 (&c)[TOK], const float4 (&s)[TOK],
                                       uint8_t *const (&to)[TOK], int apart, int kind)
{
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        float x[4], y[4], p[4], q[4];
        convert4<XT>(ra[k], x);
        convert4<XT>(rb[k], y);
        const float cc[4] = {c[k].x, c[k].y, c[k].z, c[k].w}, ss[4] = {s[k].x, s[k].y, s[k].z, s[k].w};
        if (kind == 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[j] = x[j] * cc[j] - y[j] * ss[j];
                q[j] = x[j] * ss[j] + y[j] * cc[j];
            }
        } else if (kind == 2) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                p[j] = x[j] * cc[j / 2] - x[j + 1] * ss[j / 2];
                p[j + 1] = x[j] * ss[j / 2] + x[j + 1] * cc[j / 2];
                q[j] = y[j] * cc[2 + j / 2] - y[j + 1] * ss[2 + j / 2];
                q[j + 1] = y[j] * ss[2 + j / 2] + y[j + 1] * cc[2 + j / 2];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = x[j], q[j] = y[j];
        }
        if (to[k]) {
            store4<YT>(to[k], p);
            store4<YT>(to[k] + apart * (YT == Q4K_F32 ? 4 : 2), q);
        }
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
    bool pdl;                 // launched as a programmatic dependent
    int warps;                // of a token
};

// Where a token goes and which table row turns it.
struct Place {
    int row, page, slot;
    int state;   // 0: belongs to no sequence, 1: every index is inside its buffer, 2: not so
};

template <bool APPEND>
__device__ __forceinline__ Place place_of(const TokenArgs &a, int t)
{
    Place w{0, 0, 0, 1};
    if (APPEND) {
        int b = 0, e = a.batch;   // the last sequence that starts at or before t is b - 1 or in [b, e)
        while (b < e) {
            const int m = (b + e) >> 1;
            if (a.seq_start[m] <= t) b = m + 1; else e = m;
        }
        --b;
        const int s0 = b < 0 ? 0 : a.seq_start[b], s1 = b < 0 ? 0 : a.seq_start[b + 1];
        if (t >= s1) {
            w.state = 0;
            return w;
        }
        const int64_t p = static_cast<int64_t>(a.kv_len[b]) - s1 + t;
        const int64_t row = a.rot ? (a.pos ? static_cast<int64_t>(a.pos[t]) : p) : 0;
        w.state = 2;
        if (s0 < 0 || s1 > a.tokens || p < 0 || (a.rot && (row < 0 || row >= a.table_rows))) return w;
        // (positions fit 32 bits, kv_len does)
        const uint32_t n = static_cast<uint32_t>(p) / static_cast<uint32_t>(a.page_size);
        if (n >= a.max_pages) return w;
        w.row = static_cast<int>(row);
        w.slot = static_cast<int>(static_cast<uint32_t>(p) - n * static_cast<uint32_t>(a.page_size));
        w.page = a.page_table[b * a.table_stride + n];
        if (w.page >= 0 && w.page < a.pages) w.state = 1;
    } else if (a.rot) {
        w.row = a.pos[t];
        w.state = w.row >= 0 && w.row < a.table_rows ? 1 : 2;
    }
    return w;
}

// TOK consecutive tokens per thread: their data is loaded first; then lane j of
// each warp places token j; then they are turned and stored.  HALF: all data is
// 16-bit (fewer registers, more threads).  Bound by memory latency: one token a
// thread leaves too little in flight, eight take the registers of other threads,
// and small CTAs even out the tail.  4097 tokens x 32 heads x 128 in bf16, half of
// each head turned (68 MB): 14.0 us, 4.9 TB/s (a copy of the same size takes 11.7);
// one token a thread 25 us, eight 15.8.  2048 tokens of q, k and v from fp32 (58
// MB): 14.9 us, 3.9 TB/s.
template <bool APPEND, int TOK, bool HALF>
__global__ void __launch_bounds__(kThreads, HALF ? 7 : 6) wide_kernel(const TokenArgs a)
{
    pdl_launch_dependents();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = w / a.warps;   // of TOK tokens, within the CTA
    const int i = (blockIdx.y * a.warps + (w - group * a.warps)) * 32 + lane;
    const int per = static_cast<int>(blockDim.x >> 5) / a.warps;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * per + group) * TOK;
    if (t0 >= a.tokens) return;
    const bool live = i < a.items;

    // this thread's unit: tensor, head, its two halves of four elements
    int h = (live ? i : 0) / a.units;
    const int j = (live ? i : 0) - h * a.units;
    int part = 0;
    while (h >= a.part[part].heads) h -= a.part[part].heads, ++part;
    const Part &p = a.part[part];
    const bool turned = 8 * j < p.rot, split = turned && !a.inter;
    const int ia = split ? 4 * j : 8 * j, apart = split ? p.rot >> 1 : 4;
    const int xs = p.xtype == Q4K_F32 ? 4 : 2, ys = p.ytype == Q4K_F32 ? 4 : 2;

    pdl_wait();   // (everything below may come from the kernel before)
    // (as they lie in memory: a conversion next to its load would wait for it)
    using Raw = typename std::conditional<HALF, uint2, uint4>::type;
    Raw ra[TOK], rb[TOK];
    const uint8_t *src = static_cast<const uint8_t *>(p.x) + (t0 * p.xt + h * p.xh + ia) * xs;
    const int64_t next = p.xt * xs;   // bytes to the next token
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        ra[k] = rb[k] = Raw{};
        if (live && t0 + k < a.tokens) {
            const uint8_t *q = src + k * next;
            if constexpr (HALF) {
                ra[k] = *reinterpret_cast<const uint2 *>(q), rb[k] = *reinterpret_cast<const uint2 *>(q + 2 * apart);
            } else if (xs == 4) {
                ra[k] = *reinterpret_cast<const uint4 *>(q);
                rb[k] = *reinterpret_cast<const uint4 *>(q + 4 * apart);
            } else {
                const uint2 u = *reinterpret_cast<const uint2 *>(q), v = *reinterpret_cast<const uint2 *>(q + 2 * apart);
                ra[k] = make_uint4(u.x, u.y, 0, 0), rb[k] = make_uint4(v.x, v.y, 0, 0);
            }
        }
    }

    Place mine{0, 0, 0, 0};
    if (lane < TOK && t0 + lane < a.tokens) mine = place_of<APPEND>(a, static_cast<int>(t0) + lane);
    if (mine.state == 2 && i < TOK) atomicOr(&g_rope_error, 4u);

    uint8_t *dst = static_cast<uint8_t *>(p.y) + (h * p.yh + ia) * ys;
    const float *trow = a.table + (a.inter ? ia >> 1 : ia);
    const int64_t per_page = (part ? a.v_page : a.k_page) * ys, per_slot = (part ? a.v_slot : a.k_slot) * ys;
    const int kind = !turned ? 0 : split ? 1 : 2;
    float4 c[TOK], s[TOK];
    uint8_t *to[TOK];
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const int row = __shfl_sync(0xffffffffu, mine.row, k);
        const bool good = __shfl_sync(0xffffffffu, mine.state, k) == 1 && live;
        c[k] = s[k] = make_float4(0, 0, 0, 0);
        if (good && turned) {
            const float *r = trow + static_cast<int64_t>(row) * a.rot;
            c[k] = *reinterpret_cast<const float4 *>(r);
            s[k] = *reinterpret_cast<const float4 *>(r + (a.rot >> 1));
        }
        int64_t o = (t0 + k) * p.yt * ys;
        if (APPEND) {
            const int page = __shfl_sync(0xffffffffu, mine.page, k), slot = __shfl_sync(0xffffffffu, mine.slot, k);
            if (part < 2) o = page * per_page + slot * per_slot;
        }
        to[k] = good ? dst + o : nullptr;
    }
    switch (3 * p.xtype + p.ytype) {
        case 3 * Q4K_F16 + Q4K_F32: finish<Q4K_F16, Q4K_F32, TOK>(ra, rb, c, s, to, apart, kind); break;
        case 3 * Q4K_F16 + Q4K_F16: finish<Q4K_F16, Q4K_F16, TOK>(ra, rb, c, s, to, apart, kind); break;
        case 3 * Q4K_F16 + Q4K_BF16: finish<Q4K_F16, Q4K_BF16, TOK>(ra, rb, c, s, to, apart, kind); break;
        case 3 * Q4K_BF16 + Q4K_F32: finish<Q4K_BF16, Q4K_F32, TOK>(ra, rb, c, s, to, apart, kind); break;
        case 3 * Q4K_BF16 + Q4K_F16: finish<Q4K_BF16, Q4K_F16, TOK>(ra, rb, c, s, to, apart, kind); break;
        case 3 * Q4K_BF16 + Q4K_BF16: finish<Q4K_BF16, Q4K_BF16, TOK>(ra, rb, c, s, to, apart, kind); break;
        default:
            if constexpr (!HALF) {
                if (p.ytype == Q4K_F32) finish<Q4K_F32, Q4K_F32, TOK>(ra, rb, c, s, to, apart, kind);
                else if (p.ytype == Q4K_F16) finish<Q4K_F32, Q4K_F16, TOK>(ra, rb, c, s, to, apart, kind);
                else finish<Q4K_F32, Q4K_BF16, TOK>(ra, rb, c, s, to, apart, kind);
            }
    }
}

// Element by element, for rows and sizes that the wide accesses do not fit: a
// head is its pairs, then its copied elements.
template <bool APPEND>
__global__ void __launch_bounds__(kThreads) narrow_kernel(const TokenArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int w = threadIdx.x >> 5;
    const int per = static_cast<int>(blockDim.x >> 5) / a.warps;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * per + w / a.warps;
    if (t >= a.tokens) return;
    const int first = (w % a.warps) * 32 + (threadIdx.x & 31), step = a.warps * 32;
    const Place at = place_of<APPEND>(a, static_cast<int>(t));
    if (at.state != 1) {
        if (at.state == 2 && first == 0) atomicOr(&g_rope_error, 4u);
        return;
    }
    const float *trow = a.table + static_cast<int64_t>(at.row) * a.rot;
    for (int q = 0; q < (APPEND ? 3 : 1); ++q) {
        const Part &p = a.part[q];
        const int half = p.rot >> 1, each = half + (a.dim - p.rot);
        const int64_t base = !APPEND || q == 2 ? t * p.yt
                                               : at.page * (q ? a.v_page : a.k_page) + at.slot * (q ? a.v_slot : a.k_slot);
        for (int64_t i = first; i < static_cast<int64_t>(each) * p.heads; i += step) {
            const int h = static_cast<int>(i / each), j = static_cast<int>(i - static_cast<int64_t>(h) * each);
            const int64_t from = t * p.xt + h * p.xh, to = base + h * p.yh;
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

// Warps per token, tokens per thread and CTA, then the launch.
template <bool APPEND>
static q4k_status launch_tokens(TokenArgs &a, bool wide, int sms, void *stream)
{
    int64_t heads = 0;
    for (const Part &p : a.part) heads += p.heads;
    a.units = a.dim / 8;
    const int64_t items = heads * (wide ? a.units : a.dim);
    if (items > 0x7FFFFFFF) return Q4K_ERR_INVALID_ARG;
    a.items = static_cast<int>(items);
    const int64_t need = (items + 31) / 32, rounds = (need + kThreads / 32 - 1) / (kThreads / 32);
    if (rounds > 65535) return Q4K_ERR_INVALID_ARG;
    a.warps = static_cast<int>((need + rounds - 1) / rounds);
    const int per = a.warps >= 4 ? 1 : 4 / a.warps;   // token groups of a CTA: four warps or more
    const int threads = a.warps * per * 32;
    auto grid = [&](int tok) {
        const int64_t each = static_cast<int64_t>(per) * tok;
        return dim3(static_cast<unsigned>((a.tokens + each - 1) / each), static_cast<unsigned>(wide ? rounds : 1));
    };
    auto s = static_cast<cudaStream_t>(stream);
    // several tokens a thread where one each would make 1024 threads an SM or more: us
    // of one and of four, bf16 rope of 32 heads 128 tokens 2.6 / 2.9, 256 3.2 / 2.9, 1024
    // 7.6 / 4.9; fp32 append of 28 + 8 heads 128 tokens 3.4 / 3.9, 256 4.4 / 4.4, 1024
    // 11.3 / 7.8
    const bool many = wide && static_cast<int64_t>(a.tokens) * need * 32 >= 1024LL * sms;
    bool half = true;
    for (const Part &p : a.part) half = half && (!p.heads || p.xtype != Q4K_F32);
    auto kern = !wide ? narrow_kernel<APPEND>
                : !many ? wide_kernel<APPEND, 1, false>
                : half ? wide_kernel<APPEND, kTok, true> : wide_kernel<APPEND, kTok, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid(many ? kTok : 1);
    cfg.blockDim = threads;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = a.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA;
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
        !good_type(a->x_type) || !good_type(a->y_type) || (a->interleaved & ~1) || (a->flags & ~Q4K_FLAG_PDL))
        return Q4K_ERR_INVALID_ARG;
    if (a->tokens > 0 && (!a->x || !a->y || (a->rot && (!a->pos || !a->table)))) return Q4K_ERR_INVALID_ARG;
    if (off(a->x, size_of(a->x_type)) || off(a->y, size_of(a->y_type)) || off(a->pos, 4) || off(a->table, 4))
        return Q4K_ERR_MISALIGNED;
    int sms = 0;
    q4k_status st = check_device(&sms);
    if (st != Q4K_OK || a->tokens == 0) return st;
    TokenArgs p{};
    p.part[0] = Part{a->x, a->y, used_stride(a->x_token_stride, a->tokens), used_stride(a->x_head_stride, a->heads),
                     used_stride(a->y_token_stride, a->tokens), used_stride(a->y_head_stride, a->heads),
                     static_cast<int>(a->heads), a->x_type, a->y_type, static_cast<int>(a->rot)};
    p.pos = a->pos, p.table = a->table, p.table_rows = a->table_rows;
    p.tokens = static_cast<int>(a->tokens), p.dim = static_cast<int>(a->dim), p.rot = static_cast<int>(a->rot);
    p.inter = a->interleaved, p.pdl = a->flags & Q4K_FLAG_PDL;
    const Part &r = p.part[0];
    const bool wide = a->dim % 8 == 0 && a->rot % 8 == 0 && !off(a->table, 16) &&
                      wide_rows(a->x, a->x_type, r.xt, r.xh) && wide_rows(a->y, a->y_type, r.yt, r.yh);
    return launch_tokens<false>(p, wide, sms, stream);
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

q4k_paged_cache with_used_strides(q4k_paged_cache c)
{
    c.k_page_stride = used_stride(c.k_page_stride, c.pages), c.v_page_stride = used_stride(c.v_page_stride, c.pages);
    c.k_slot_stride = used_stride(c.k_slot_stride, c.page_size), c.v_slot_stride = used_stride(c.v_slot_stride, c.page_size);
    c.k_head_stride = used_stride(c.k_head_stride, c.heads), c.v_head_stride = used_stride(c.v_head_stride, c.heads);
    return c;
}

q4k_status kv_append_impl(const q4k_paged_cache *c, const q4k_append_args *a, void *stream)
{
    using namespace rope;
    q4k_status st = check_cache(c);
    if (st == Q4K_ERR_INVALID_ARG || !a) return Q4K_ERR_INVALID_ARG;
    const q4k_paged_cache used = with_used_strides(*c);
    c = &used;
    const bool some = c->tokens > 0 && c->batch > 0;
    if (a->rot < 0 || a->rot % 2 || a->rot > c->dim || a->rot > kMaxRot || a->table_rows < 0 ||
        !good_type(a->kv_type) || (a->interleaved & ~1) || (a->flags & ~Q4K_FLAG_PDL) || (a->q == nullptr) != (a->q_out == nullptr))
        return Q4K_ERR_INVALID_ARG;
    if (a->q && (a->q_heads < 1 || a->q_heads > 65536 || !good_type(a->q_type) || !good_type(a->q_out_type)))
        return Q4K_ERR_INVALID_ARG;
    if (some && (!a->k || !a->v || (a->rot && !a->table))) return Q4K_ERR_INVALID_ARG;
    if (st != Q4K_OK) return st;
    if (off(a->k, size_of(a->kv_type)) || off(a->v, size_of(a->kv_type)) || off(a->pos, 4) || off(a->table, 4) ||
        (a->q && (off(a->q, size_of(a->q_type)) || off(a->q_out, size_of(a->q_out_type)))))
        return Q4K_ERR_MISALIGNED;
    int sms = 0;
    st = check_device(&sms);
    if (st != Q4K_OK || !some) return st;
    TokenArgs p{};
    const int heads = static_cast<int>(c->heads), rot = static_cast<int>(a->rot);
    const int64_t n = c->tokens;
    p.part[0] = Part{a->k, c->k, used_stride(a->k_token_stride, n), used_stride(a->k_head_stride, heads), 0, c->k_head_stride,
                     heads, a->kv_type, c->type, rot};
    p.part[1] = Part{a->v, c->v, used_stride(a->v_token_stride, n), used_stride(a->v_head_stride, heads), 0, c->v_head_stride,
                     heads, a->kv_type, c->type, 0};
    if (a->q)
        p.part[2] = Part{a->q, a->q_out, used_stride(a->q_token_stride, n), used_stride(a->q_head_stride, a->q_heads),
                         used_stride(a->q_out_token_stride, n), used_stride(a->q_out_head_stride, a->q_heads),
                         static_cast<int>(a->q_heads), a->q_type, a->q_out_type, rot};
    p.k_page = c->k_page_stride, p.k_slot = c->k_slot_stride, p.v_page = c->v_page_stride, p.v_slot = c->v_slot_stride;
    p.pages = c->pages, p.page_size = c->page_size, p.table_stride = c->page_table_stride, p.max_pages = c->max_pages;
    p.page_table = c->page_table, p.seq_start = c->seq_start, p.kv_len = c->kv_len, p.pos = a->pos;
    p.table = a->table, p.table_rows = a->table_rows;
    p.batch = static_cast<int>(c->batch), p.tokens = static_cast<int>(c->tokens), p.dim = static_cast<int>(c->dim);
    p.rot = rot, p.inter = a->interleaved, p.pdl = a->flags & Q4K_FLAG_PDL;
    const Part &k = p.part[0], &v = p.part[1], &q = p.part[2];
    bool wide = c->dim % 8 == 0 && rot % 8 == 0 && !off(a->table, 16) && wide_rows(a->k, a->kv_type, k.xt, k.xh) &&
                wide_rows(a->v, a->kv_type, v.xt, v.xh) && wide_rows(c->k, c->type, p.k_page, p.k_slot) &&
                wide_rows(c->v, c->type, p.v_page, p.v_slot) && k.yh % 8 == 0 && v.yh % 8 == 0;
    if (a->q) wide = wide && wide_rows(a->q, a->q_type, q.xt, q.xh) && wide_rows(a->q_out, a->q_out_type, q.yt, q.yh);
    return launch_tokens<true>(p, wide, sms, stream);
}

}  // namespace q4k
