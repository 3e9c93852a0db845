// q4k_cache8.cu -- head norms with the rotation in the same pass (q4k_norm_rope),
// the append of keys and values to a paged cache in 8 bits (q4k_kv_append8) and the
// way back (q4k_kv_read8).
//
// Bound by memory, or for a few tokens by the chain of dependent index loads.  A
// head of a token is E = 8 pairs a lane where dim and rot are multiples of 16 (8 lanes up
// to a dim of 128, 16 above), else 4; a warp holds several such rows in registers, all
// loaded before the index chain begins.  (4 pairs a lane throughout: 39 us for 4097
// tokens of 40 heads, half of each turned.)
// The norm is one sum over a lane group; pairs turn in the lane that holds them.
//
// Measured (device): norms of 4097 tokens of 40 bf16 heads, half of each turned, 26.9 us
// (85 MB; the rotation alone moves as much in 18), bound by issue slots and latency alike
// (6 CTAs of 128 threads an SM; 5: 31 us, 8: 29); three prompts of 2500 tokens, 32 / 8 bf16
// heads, appended 47 us (queries in a launch of their own: no less) and read back 13; 65536
// positions of 8 heads read to bf16 76 us, 5.3 TB/s.  One token: 4 to 6 us of launch and
// index loads.
//
// Quantising: a warp (several for blocks of more tokens than it holds) takes an
// aligned run of positions of one head, so that every block lies in one warp, or in
// the warps of one CTA: max|x| over the lanes, the rows and the warps, one scale, one
// store of codes.  Nothing is read twice and nothing is written that another warp
// decides, so no atomics and no second launch.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/q4k.h"
#include "ptx.cuh"
#include "q4k_attn.cuh"
#include "q4k_cache8.cuh"
#include "q4k_internal.h"

namespace q4k {

__device__ unsigned int g_cache8_error = 0;   // bit 2: an index outside its buffer

unsigned int read_cache8_error()
{
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_cache8_error, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
    return v;
}

bool clear_cache8_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_cache8_error, &z, sizeof(z)) == cudaSuccess;
}

namespace cache8 {

constexpr int kMaxRot = 512, kMaxDim = 256;
constexpr int rows_of(int e) { return 32 / e; }   // rows of a lane group that a warp of the cache's side holds
constexpr int kWarps = 4;        // of a CTA where one warp holds a block
constexpr int kMaxBlock = 128;   // tokens of a scale
constexpr int kMaxWarps = kMaxBlock / 8;

// One tensor of heads.
struct Heads {
    const void *x;
    void *y;
    const float *weight;                    // (or null)
    int64_t xt, xh, yt, yh, wh;             // strides in elements
    int heads, xtype, ytype;
    int rot;                                // turned elements of a head (0: none)
};

// Where tokens are.
struct Index {
    const int32_t *page_table, *seq_start, *kv_len, *pos;
    int64_t pages, table_stride, max_pages, table_rows;
    int page_size, batch, tokens;
};

struct Args {
    Heads q, k, v;          // norm_rope: q and k; append: v too (y of k and v unused); read: y of k and v
    Index at;
    const float *table;
    uint8_t *kc, *vc;       // codes
    float *ks, *vs;         // scales
    int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
    int64_t ks_page, ks_block, ks_head, vs_page, vs_block, vs_head;
    int dim, rot, inter, codes;
    int block, shift;       // tokens of a scale, its log2
    int lanes;              // of a row: a power of two, dim / (2 E) of them at least
    float over_dim;         // 1 / dim
    int run, warps;         // append: positions of an item, warps that hold them
    int slots;              // append: items of a head and tensor at most
    int kv_ctas;            // append: CTAs of the cache's side, the queries' follow
    float eps;
    bool pdl;
};

// ---------------------------------------------------------------- a row's pairs

// A lane's pairs of a head: pair j is (a[j], b[j]).
template <int E>
struct Pairs {
    float a[E], b[E];
};

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

// Where a lane's pairs lie in a head.  Turned pairs are (p, p + rot/2), or (2p, 2p + 1)
// if INTER; what is not turned goes alike, in halves or in neighbours, so that every lane
// does the same.  Wide accesses (rot and dim multiples of 2 E) take E elements at `ia`, E
// at `ib`, each from neighbouring lanes without gaps (16 bytes of every 32 in two turns
// took 33 us where this takes 31).  Pair j has the table's entry pa + j, for INTER from
// the second half of the pairs on pb + j - E/2.  (Narrow accesses: pair E u + j.)
template <int E, bool INTER>
struct Lane {
    int u;                  // unit
    bool live, turned, turned_b;   // (turned_b: INTER, of the pairs of ib)
    int ia, ib, pa, pb;

    __device__ __forceinline__ Lane(const Args &a, int rot, int lane) : u(lane & (a.lanes - 1))
    {
        live = 2 * E * u < a.dim;
        if constexpr (INTER) {
            ia = E * u, ib = E * u + (a.dim >> 1);
            turned = ia < rot, turned_b = ib < rot;
            pa = ia >> 1, pb = ib >> 1;
        } else {
            turned = turned_b = 2 * E * u < rot;
            const int rest = rot + E * u - (rot >> 1);   // of the units behind the turned ones
            ia = turned ? E * u : rest;
            ib = turned ? E * u + (rot >> 1) : rest + ((a.dim - rot) >> 1);
            pa = E * u, pb = pa + E / 2;
        }
    }
};

// Elements of pair p, for any even rot.
__device__ __forceinline__ void pair_at(int p, int rot, int inter, int &i, int &j)
{
    if (2 * p < rot && !inter) i = p, j = p + (rot >> 1);
    else i = 2 * p, j = i + 1;
}

// E elements at ia and E at ib as pairs, and back.
template <int E, bool INTER>
__device__ __forceinline__ void arrange(const float (&x)[E], const float (&y)[E], Pairs<E> &r)
{
#pragma unroll
    for (int j = 0; j < E; ++j) {
        if constexpr (INTER) r.a[j] = j < E / 2 ? x[2 * j & (E - 1)] : y[2 * j & (E - 1)], r.b[j] = j < E / 2 ? x[(2 * j & (E - 1)) + 1] : y[(2 * j & (E - 1)) + 1];
        else r.a[j] = x[j], r.b[j] = y[j];
    }
}

template <int E, bool INTER>
__device__ __forceinline__ void disarrange(const Pairs<E> &r, float (&x)[E], float (&y)[E])
{
#pragma unroll
    for (int j = 0; j < E; ++j) {
        if constexpr (INTER) x[j] = j & 1 ? r.b[j / 2] : r.a[j / 2], y[j] = j & 1 ? r.b[E / 2 + j / 2] : r.a[E / 2 + j / 2];
        else x[j] = r.a[j], y[j] = r.b[j];
    }
}

// E elements in one access (16 bits) or E / 4 (fp32).
template <int E>
struct Raw16 {
    uint2 v[E / 4];
};
template <int E>
__device__ __forceinline__ Raw16<E> load16(const uint16_t *p)
{
    Raw16<E> r;
    if constexpr (E == 8) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        r.v[0] = make_uint2(x.x, x.y), r.v[1] = make_uint2(x.z, x.w);
    } else {
        r.v[0] = *reinterpret_cast<const uint2 *>(p);
    }
    return r;
}

template <int E>
__device__ __forceinline__ void unpack(const Raw16<E> &r, int type, float (&f)[E])
{
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
        const float2 a = attn::unpack2(r.v[j].x, type), b = attn::unpack2(r.v[j].y, type);
        f[4 * j] = a.x, f[4 * j + 1] = a.y, f[4 * j + 2] = b.x, f[4 * j + 3] = b.y;
    }
}

// N rows of a lane group, the first at element `base`, `step` elements apart;
// row k where `there` has bit k.  All loads first, conversions after.
template <bool WIDE, int N, int E, bool INTER>
__device__ __forceinline__ void load_rows(const void *x, int type, int64_t base, int64_t step, const Lane<E, INTER> &l, int rot, int inter,
                                          uint32_t there, Pairs<E> (&r)[N])
{
    if constexpr (WIDE) {
        if (type == Q4K_F32) {
            float p[N][E], q[N][E];
            const float *s = static_cast<const float *>(x) + base;
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int j = 0; j < E; j += 4) {
                    float4 v = make_float4(0, 0, 0, 0), z = v;
                    if (there >> k & 1) {
                        v = *reinterpret_cast<const float4 *>(s + k * step + l.ia + j);
                        z = *reinterpret_cast<const float4 *>(s + k * step + l.ib + j);
                    }
                    p[k][j] = v.x, p[k][j + 1] = v.y, p[k][j + 2] = v.z, p[k][j + 3] = v.w;
                    q[k][j] = z.x, q[k][j + 1] = z.y, q[k][j + 2] = z.z, q[k][j + 3] = z.w;
                }
#pragma unroll
            for (int k = 0; k < N; ++k) arrange<E, INTER>(p[k], q[k], r[k]);
        } else {
            Raw16<E> p[N], q[N];
            const uint16_t *s = static_cast<const uint16_t *>(x) + base;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                p[k] = q[k] = Raw16<E>{};
                if (there >> k & 1) p[k] = load16<E>(s + k * step + l.ia), q[k] = load16<E>(s + k * step + l.ib);
            }
            auto all = [&](auto t) {   // (the type outside the rows)
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    float a[E], b[E];
                    unpack<E>(p[k], decltype(t)::value, a);
                    unpack<E>(q[k], decltype(t)::value, b);
                    arrange<E, INTER>(a, b, r[k]);
                }
            };
            if (type == Q4K_F16) all(std::integral_constant<int, Q4K_F16>{});
            else all(std::integral_constant<int, Q4K_BF16>{});
        }
    } else {
#pragma unroll 1
        for (int k = 0; k < N; ++k) {
            Pairs<E> one;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                int c, d;
                pair_at(E * l.u + j, rot, inter, c, d);
                one.a[j] = one.b[j] = 0.0f;
                if (there >> k & 1) one.a[j] = load1(x, type, base + k * step + c), one.b[j] = load1(x, type, base + k * step + d);
            }
#pragma unroll
            for (int m = 0; m < N; ++m)   // (registers have no run-time index)
                if (m == k) r[m] = one;
        }
    }
}

template <bool WIDE, int E, bool INTER>
__device__ __forceinline__ void store_row(void *y, int type, int64_t base, const Lane<E, INTER> &l, int rot, int inter, const Pairs<E> &r)
{
    if constexpr (WIDE) {
        float a[E], b[E];
        disarrange<E, INTER>(r, a, b);
        if (type == Q4K_F32) {
            float *d = static_cast<float *>(y) + base;
#pragma unroll
            for (int j = 0; j < E; j += 4) {
                *reinterpret_cast<float4 *>(d + l.ia + j) = make_float4(a[j], a[j + 1], a[j + 2], a[j + 3]);
                *reinterpret_cast<float4 *>(d + l.ib + j) = make_float4(b[j], b[j + 1], b[j + 2], b[j + 3]);
            }
        } else {
            uint16_t *d = static_cast<uint16_t *>(y) + base;
            uint32_t p[E / 2], q[E / 2];
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                p[j] = attn::pack2(a[2 * j], a[2 * j + 1], type);
                q[j] = attn::pack2(b[2 * j], b[2 * j + 1], type);
            }
            if constexpr (E == 8) {
                *reinterpret_cast<uint4 *>(d + l.ia) = make_uint4(p[0], p[1], p[2], p[3]);
                *reinterpret_cast<uint4 *>(d + l.ib) = make_uint4(q[0], q[1], q[2], q[3]);
            } else {
                *reinterpret_cast<uint2 *>(d + l.ia) = make_uint2(p[0], p[1]);
                *reinterpret_cast<uint2 *>(d + l.ib) = make_uint2(q[0], q[1]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            int c, d;
            pair_at(E * l.u + j, rot, inter, c, d);
            store1(y, type, base + c, r.a[j]);
            store1(y, type, base + d, r.b[j]);
        }
    }
}

// A lane's weights, ones where there are none.
template <bool WIDE, int E, bool INTER>
__device__ __forceinline__ void load_weight(const Heads &h, int head, const Lane<E, INTER> &l, int inter, Pairs<E> &w)
{
#pragma unroll
    for (int j = 0; j < E; ++j) w.a[j] = w.b[j] = 1.0f;
    if (!h.weight || !l.live) return;
    Pairs<E> one[1];
    load_rows<WIDE, 1, E, INTER>(h.weight, Q4K_F32, head * h.wh, 0, l, h.rot, inter, 1u, one);
    w = one[0];
}

// Sum and maximum over a row's lanes; whole warps.
__device__ __forceinline__ float row_sum(float s, int lanes)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < lanes) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Normed in place; whole warps.
template <int E>
__device__ __forceinline__ void norm(Pairs<E> &r, const Pairs<E> &w, int lanes, float over_dim, float eps)
{
    float s = 0.0f, z = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) s = fmaf(r.a[j], r.a[j], s), z = fmaf(r.b[j], r.b[j], z);
    const float f = 1.0f / sqrtf(fmaf(row_sum(s + z, lanes), over_dim, eps));
#pragma unroll
    for (int j = 0; j < E; ++j) r.a[j] *= f * w.a[j], r.b[j] *= f * w.b[j];
}

// A lane's cosines and sines in a table row, and a turn by them.
template <int E>
struct Turn {
    float c[E], s[E];
};
template <bool WIDE, int E, bool INTER>
__device__ __forceinline__ void load_turn(Turn<E> &t, const float *row, const Lane<E, INTER> &l, int rot)
{
    if constexpr (WIDE && E == 8) {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
            if (!(j ? l.turned_b : l.turned)) continue;
            const float *p = row + (j ? l.pb : l.pa);
            const float4 c = *reinterpret_cast<const float4 *>(p), s = *reinterpret_cast<const float4 *>(p + (rot >> 1));
            t.c[j] = c.x, t.c[j + 1] = c.y, t.c[j + 2] = c.z, t.c[j + 3] = c.w;
            t.s[j] = s.x, t.s[j + 1] = s.y, t.s[j + 2] = s.z, t.s[j + 3] = s.w;
        }
    } else if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < E; j += 2) {   // (E = 4: two pairs of each part)
            if (!(j ? l.turned_b : l.turned)) continue;
            const float *p = row + (j ? l.pb : l.pa);
            const float2 c = *reinterpret_cast<const float2 *>(p), s = *reinterpret_cast<const float2 *>(p + (rot >> 1));
            t.c[j] = c.x, t.c[j + 1] = c.y, t.s[j] = s.x, t.s[j + 1] = s.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int p = E * l.u + j;
            if (2 * p < rot) t.c[j] = row[p], t.s[j] = row[(rot >> 1) + p];
        }
    }
}
template <bool WIDE, int E, bool INTER>
__device__ __forceinline__ void turn(Pairs<E> &r, const Turn<E> &t, const Lane<E, INTER> &l, int rot)
{
#pragma unroll
    for (int j = 0; j < E; ++j) {
        if (WIDE ? !(j < E / 2 ? l.turned : l.turned_b) : 2 * (E * l.u + j) >= rot) continue;
        const float x = r.a[j], y = r.b[j];
        r.a[j] = x * t.c[j] - y * t.s[j];
        r.b[j] = x * t.s[j] + y * t.c[j];
    }
}

// ---------------------------------------------------------------- where tokens are

struct Place {
    int row, page, slot;
    int state;   // 0: belongs to no sequence, 1: every index is inside its buffer, 2: not so
};

__device__ __forceinline__ int start_of(const Index &x, int b) { return min(max(x.seq_start[b], 0), x.tokens); }

// Page and slot of position p of sequence b, and the table row of token row t there.
__device__ __forceinline__ Place place_at(const Args &a, int b, int64_t p, int t, int rot)
{
    Place w{0, 0, 0, 2};
    const int64_t row = rot ? (a.at.pos ? static_cast<int64_t>(a.at.pos[t]) : p) : 0;
    if (p < 0 || (rot && (row < 0 || row >= a.at.table_rows))) return w;
    const uint32_t n = static_cast<uint32_t>(p) / static_cast<uint32_t>(a.at.page_size);   // (positions fit 32 bits, kv_len does)
    if (n >= a.at.max_pages) return w;
    w.row = static_cast<int>(row);
    w.slot = static_cast<int>(static_cast<uint32_t>(p) - n * static_cast<uint32_t>(a.at.page_size));
    w.page = a.at.page_table[b * a.at.table_stride + n];
    if (w.page >= 0 && w.page < a.at.pages) w.state = 1;
    return w;
}

// The place of token row t.
__device__ __forceinline__ Place place_of(const Args &a, int t, int rot)
{
    int b = 0, e = a.at.batch;   // the last sequence that starts at or before t is b - 1 or in [b, e)
    while (b < e) {
        const int m = (b + e) >> 1;
        if (a.at.seq_start[m] <= t) b = m + 1; else e = m;
    }
    --b;
    const int s0 = b < 0 ? 0 : a.at.seq_start[b], s1 = b < 0 ? 0 : a.at.seq_start[b + 1];
    if (t >= s1) return Place{0, 0, 0, 0};
    if (s0 < 0 || s1 > a.at.tokens) return Place{0, 0, 0, 2};
    return place_at(a, b, static_cast<int64_t>(a.at.kv_len[b]) - s1 + t, t, rot);
}

// ---------------------------------------------------------------- queries (and norm_rope's keys)

// Heads of a chunk: N rows a lane group of one token.
__host__ __device__ __forceinline__ int chunk_heads(int n, int lanes) { return n * (32 / lanes); }

// A chunk of a token's heads from head0 on: normed, turned, stored.  APPEND: the token is
// placed by its sequence, else by pos.  (Heads of one token lie together and share its
// table row; rows of one head of several tokens took 31 us where this takes 27.)
template <bool WIDE, int N, int E, bool INTER, bool APPEND>
__device__ __forceinline__ void turn_rows(const Args &a, const Heads &h, int head0, int64_t t)
{
    const int lane = threadIdx.x & 31, groups = 32 / a.lanes, first = head0 + lane / a.lanes;
    const Lane<E, INTER> l(a, h.rot, lane);
    // row k of this group: head first + k groups
    uint32_t there = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (l.live && first + k * groups < h.heads) there |= 1u << k;
    Pairs<E> r[N];
    Place at{0, 0, 0, 1};
    if (!APPEND && h.rot) {   // (one load: ahead of the data; the append's chain of them behind it)
        at.row = a.at.pos[t];
        if (at.row < 0 || at.row >= a.at.table_rows) at.state = 2;
    }
    load_rows<WIDE, N, E, INTER>(h.x, h.xtype, t * h.xt + first * h.xh, groups * h.xh, l, h.rot, a.inter, there, r);
    if (APPEND) at = place_of(a, static_cast<int>(t), h.rot);
    if (at.state == 2 && lane == 0) atomicOr(&g_cache8_error, 4u);
    if (at.state != 1) return;   // (the whole warp)
    Turn<E> by;
    if (h.rot) load_turn<WIDE, E, INTER>(by, a.table + static_cast<int64_t>(at.row) * a.rot, l, h.rot);
    if (h.weight) {
        Pairs<E> w;
        if (!h.wh) load_weight<WIDE, E, INTER>(h, 0, l, a.inter, w);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (h.wh) load_weight<WIDE, E, INTER>(h, min(first + k * groups, h.heads - 1), l, a.inter, w);
            norm<E>(r[k], w, a.lanes, a.over_dim, a.eps);
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (!(there >> k & 1)) continue;
        if (h.rot) turn<WIDE, E, INTER>(r[k], by, l, h.rot);
        store_row<WIDE, E, INTER>(h.y, h.ytype, t * h.yt + (first + k * groups) * h.yh, l, h.rot, a.inter, r[k]);
    }
}

template <bool WIDE, int N, int E, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, N * E == 16 ? 6 : 8) norm_rope_kernel(const __grid_constant__ Args a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int per = chunk_heads(N, a.lanes), of_q = (a.q.heads + per - 1) / per, chunks = of_q + (a.k.heads + per - 1) / per;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), t = attn::quotient(item, chunks);
    if (t >= a.at.tokens) return;
    const int c = static_cast<int>(item - t * chunks);
    const bool keys = c >= of_q;
    turn_rows<WIDE, N, E, INTER, false>(a, keys ? a.k : a.q, (keys ? c - of_q : c) * per, t);
}

// ---------------------------------------------------------------- the cache's side of an append

// Codes of a lane's pairs, times inv.
template <bool WIDE, int E, bool INTER>
__device__ __forceinline__ void store_codes(uint8_t *to, int codes, const Lane<E, INTER> &l, int rot, int inter, const Pairs<E> &r, float inv)
{
    float x[E], y[E];
    if constexpr (WIDE) disarrange<E, INTER>(r, x, y);
    else {
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = r.a[j], y[j] = r.b[j];
    }
    uint32_t p[E / 4], q[E / 4];
#pragma unroll
    for (int j = 0; j < E; j += 4) {
        const float f[4] = {x[j] * inv, x[j + 1] * inv, x[j + 2] * inv, x[j + 3] * inv};
        const float z[4] = {y[j] * inv, y[j + 1] * inv, y[j + 2] * inv, y[j + 3] * inv};
        p[j / 4] = encode4(f, codes), q[j / 4] = encode4(z, codes);
    }
    if constexpr (WIDE && E == 8) {
        *reinterpret_cast<uint2 *>(to + l.ia) = make_uint2(p[0], p[1]);
        *reinterpret_cast<uint2 *>(to + l.ib) = make_uint2(q[0], q[1]);
    } else if constexpr (WIDE) {
        *reinterpret_cast<uint32_t *>(to + l.ia) = p[0];
        *reinterpret_cast<uint32_t *>(to + l.ib) = q[0];
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            int c, d;
            pair_at(E * l.u + j, rot, inter, c, d);
            to[c] = static_cast<uint8_t>(p[j / 4] >> 8 * (j & 3));
            to[d] = static_cast<uint8_t>(q[j / 4] >> 8 * (j & 3));
        }
    }
}

// The older codes of a block, from one scale to another (ratio of the two).
template <int E, bool INTER>
__device__ __forceinline__ void scale_codes(uint8_t *at, int codes, float ratio, const Lane<E, INTER> &l)
{
#pragma unroll 1
    for (int h = 0; h < 2 * E; h += 4) {
        uint32_t w = 0;   // (bytes: rows may start anywhere)
#pragma unroll
        for (int j = 0; j < 4; ++j) w |= static_cast<uint32_t>(at[2 * E * l.u + h + j]) << 8 * j;
        float f[4];
        decode4(w, codes, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] *= ratio;
        w = encode4(f, codes);
#pragma unroll
        for (int j = 0; j < 4; ++j) at[2 * E * l.u + h + j] = static_cast<uint8_t>(w >> 8 * j);
    }
}

// An aligned run of positions of one sequence, head and tensor.
template <bool WIDE, int E, bool INTER>
__device__ __forceinline__ void append_run(const Args &a, float *s_max)
{
    constexpr int kRows = rows_of(E);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, groups = 32 / a.lanes, g = lane / a.lanes, hold = kRows * groups;
    const int per = static_cast<int>(blockDim.x >> 5) / a.warps;   // items of a CTA
    const int64_t item = static_cast<int64_t>(blockIdx.x) * per + w / a.warps;
    const int both = 2 * a.k.heads;
    const int64_t slot = attn::quotient(item, both);
    int head = static_cast<int>(item - slot * both);
    const bool values = head >= a.k.heads;
    if (values) head -= a.k.heads;
    const Heads &h = values ? a.v : a.k;

    // the run's sequence: slots 2 b and 2 b + 1 are sequence b's first two runs, the
    // others take the slots from 2 batch + start / run on, which has room for them
    int b = 0, j = 0;
    bool any = slot < a.slots;
    if (any) {
        if (slot < 2 * a.at.batch) {
            b = static_cast<int>(slot >> 1), j = static_cast<int>(slot & 1);
        } else {
            const int x = static_cast<int>(slot) - 2 * a.at.batch;
            int e = a.at.batch - 1;
            while (b < e) {   // the last sequence with start / run <= x
                const int m = (b + e + 1) >> 1;
                if (start_of(a.at, m) / a.run <= x) b = m; else e = m - 1;
            }
            j = x - start_of(a.at, b) / a.run + 2;
            any = j >= 2;
        }
    }
    int s0 = 0, s1 = 0, len = 0;
    if (any) {
        s0 = a.at.seq_start[b], s1 = a.at.seq_start[b + 1], len = a.at.kv_len[b];
        any = s1 > s0;
        if (any && (s0 < 0 || s1 > a.at.tokens || len < s1 - s0)) {   // (a length that does not hold the new tokens)
            if (lane == 0) atomicOr(&g_cache8_error, 4u);
            any = false;
        }
    }
    const int64_t p0 = any ? static_cast<int64_t>(len) - (s1 - s0) : 0;   // the first new position
    // this warp's positions
    const int64_t base = any ? (p0 / a.run + j) * a.run + (w % a.warps) * hold : 0;
    const bool here = any && base < len && ((base + hold - 1) >> a.shift) >= (p0 >> a.shift);   // (older tokens of its block count)
    const Lane<E, INTER> l(a, h.rot, lane);
    uint32_t there = 0;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t p = base + k * groups + g;
        if (here && l.live && p >= p0 && p < len) there |= 1u << k;
    }
    Pairs<E> r[kRows], wt;
    const int64_t first = s0 + (base - p0) + g;   // token row of this group's first position
    load_rows<WIDE, kRows, E, INTER>(h.x, h.xtype, first * h.xt + head * h.xh, groups * h.xt, l, h.rot, a.inter, there, r);
    load_weight<WIDE, E, INTER>(h, head, l, a.inter, wt);
    // lane i places position base + i, the block's older ones too
    Place mine{0, 0, 0, 0};
    const int64_t p = base + lane;
    const bool older = here && lane < hold && p < p0 && (p >> a.shift) == (p0 >> a.shift);
    if (here && lane < hold && (older || (p >= p0 && p < len)))
        mine = place_at(a, b, p, older ? s0 : static_cast<int>(s0 + (p - p0)), older ? 0 : h.rot);
    if (mine.state == 2) atomicOr(&g_cache8_error, 4u);

    float most[kRows];
    uint32_t good = 0;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int from = k * groups + g;
        const int row = __shfl_sync(0xffffffffu, mine.row, from), state = __shfl_sync(0xffffffffu, mine.state, from);
        if (h.weight) norm<E>(r[k], wt, a.lanes, a.over_dim, a.eps);
        most[k] = -1.0f;   // (a block without a token that has a place stays as it is)
        if (state == 1 && (there >> k & 1)) {
            good |= 1u << k;
            most[k] = 0.0f;
            if (h.rot) {
                Turn<E> by;
                load_turn<WIDE, E, INTER>(by, a.table + static_cast<int64_t>(row) * a.rot, l, h.rot);
                turn<WIDE, E, INTER>(r[k], by, l, h.rot);
            }
#pragma unroll
            for (int z = 0; z < E; ++z) most[k] = fmaxf(most[k], fmaxf(finite_size(r[k].a[z]), finite_size(r[k].b[z])));
        }
    }
    // over a row's lanes, then over the rows of a block: lane groups, rows, warps
    // (lane groups hold neighbouring positions: those of a block are the first of them that matter)
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        if (o < a.lanes || (o < 32 && o / a.lanes < a.block)) {
#pragma unroll
            for (int k = 0; k < kRows; ++k) most[k] = fmaxf(most[k], __shfl_xor_sync(0xffffffffu, most[k], o));
        }
    }
#pragma unroll
    for (int step = 1; step < kRows; step <<= 1) {
        if (a.block > step * groups) {
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                if (!(k & step)) most[k] = most[k | step] = fmaxf(most[k], most[k | step]);
        }
    }
    if (a.warps > 1) {
        if (lane == 0) s_max[w] = most[0];
        __syncthreads();
        float m = -1.0f;
        for (int z = 0; z < a.warps; ++z) m = fmaxf(m, s_max[w - w % a.warps + z]);
#pragma unroll
        for (int k = 0; k < kRows; ++k) most[k] = m;
    }

    uint8_t *codes = values ? a.vc : a.kc;
    float *scales = values ? a.vs : a.ks;
    const int64_t c_page = values ? a.v_page : a.k_page, c_slot = values ? a.v_slot : a.k_slot, c_head = values ? a.v_head : a.k_head;
    const int64_t s_page = values ? a.vs_page : a.ks_page, s_block = values ? a.vs_block : a.ks_block,
                  s_head = values ? a.vs_head : a.ks_head;
    auto scale_at = [&](int page, int sl) { return scales + page * s_page + (sl >> a.shift) * s_block + head * s_head; };
    // the old scale of the block that holds the first new position, read by every
    // warp of the block before one of them writes the new one
    float before = 0.0f;
    const bool mixed = here && (p0 & (a.block - 1)) != 0 && (base >> a.shift) <= (p0 >> a.shift);   // (this warp may hold part of it)
    const bool of_first = (p >> a.shift) == (p0 >> a.shift);
    const int one = __ffs(__ballot_sync(0xffffffffu, mixed && of_first && mine.state == 1)) - 1;
    if (one >= 0) before = *scale_at(__shfl_sync(0xffffffffu, mine.page, one), __shfl_sync(0xffffffffu, mine.slot, one));
    __syncwarp();
    if (a.warps > 1) __syncthreads();
    const float top = top_of(a.codes);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int from = k * groups + g;
        const int page = __shfl_sync(0xffffffffu, mine.page, from), sl = __shfl_sync(0xffffffffu, mine.slot, from);
        const int state = __shfl_sync(0xffffffffu, mine.state, from);
        const int64_t q = base + from;
        const bool in_first = mixed && (q >> a.shift) == (p0 >> a.shift);
        float s = fmaxf(most[k] / top, kLeastScale);
        if (in_first) s = fmaxf(s, fabsf(before));   // (a negative one: the older codes take its sign)
        const float inv = 1.0f / s;
        uint8_t *to = codes + page * c_page + sl * c_slot + head * c_head;
        if (good >> k & 1) {
            store_codes<WIDE, E, INTER>(to, a.codes, l, h.rot, a.inter, r[k], inv);
            // (every token of a block writes the same scale: which of them have a place differs)
            if (l.u == 0) *scale_at(page, sl) = s;
        } else if (in_first && q < p0 && state == 1 && l.live && most[k] >= 0.0f && s != before) {
            scale_codes<E, INTER>(to, a.codes, before * inv, l);
        }
    }
}

// FIVE: 96 registers instead of 128, five CTAs of 128 threads an SM instead of four.
template <bool WIDE, int N, int E, bool INTER, bool FIVE>
__global__ void __launch_bounds__(FIVE ? 640 : kMaxWarps * 32) append8_kernel(const __grid_constant__ Args a)
{
    __shared__ float s_max[kMaxWarps];
    pdl_launch_dependents();
    pdl_wait();
    if (static_cast<int>(blockIdx.x) < a.kv_ctas) {
        append_run<WIDE, E, INTER>(a, s_max);
        return;
    }
    const int64_t item = static_cast<int64_t>(blockIdx.x - a.kv_ctas) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int per = chunk_heads(N, a.lanes), chunks = (a.q.heads + per - 1) / per;
    const int64_t t = attn::quotient(item, chunks);
    if (t < a.at.tokens) turn_rows<WIDE, N, E, INTER, true>(a, a.q, static_cast<int>(item - t * chunks) * per, t);
}

// ---------------------------------------------------------------- reading back

// A warp: kRows rows a lane group of one head and tensor, 8 codes a lane.
template <bool WIDE>
__global__ void __launch_bounds__(kWarps * 32) read8_kernel(const __grid_constant__ Args a)
{
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kRows = 8;
    const int lane = threadIdx.x & 31, groups = 32 / a.lanes, g = lane / a.lanes, u = lane % a.lanes, hold = kRows * groups;
    const int heads = a.k.heads + a.v.heads;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t group = attn::quotient(item, heads), t0 = group * hold;
    int head = static_cast<int>(item - group * heads);
    if (t0 >= a.at.tokens) return;
    const bool values = head >= a.k.heads, live = 8 * u < a.dim;
    if (values) head -= a.k.heads;
    const Heads &h = values ? a.v : a.k;
    const uint8_t *codes = (values ? a.vc : a.kc) + head * (values ? a.v_head : a.k_head);
    const float *scales = (values ? a.vs : a.ks) + head * (values ? a.vs_head : a.ks_head);
    const int64_t c_page = values ? a.v_page : a.k_page, c_slot = values ? a.v_slot : a.k_slot;
    const int64_t s_page = values ? a.vs_page : a.ks_page, s_block = values ? a.vs_block : a.ks_block;
    Place mine{0, 0, 0, 0};
    if (lane < hold && t0 + lane < a.at.tokens) mine = place_of(a, static_cast<int>(t0) + lane, 0);
    if (mine.state == 2) atomicOr(&g_cache8_error, 4u);
    uint2 c[kRows];
    float s[kRows];
    uint32_t good = 0;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int from = k * groups + g;
        const int64_t page = __shfl_sync(0xffffffffu, mine.page, from);
        const int slot = __shfl_sync(0xffffffffu, mine.slot, from), state = __shfl_sync(0xffffffffu, mine.state, from);
        c[k] = make_uint2(0, 0), s[k] = 0.0f;
        if (state == 1 && live) {
            good |= 1u << k;
            const uint8_t *p = codes + page * c_page + slot * c_slot + 8 * u;
            if constexpr (WIDE) {
                c[k] = *reinterpret_cast<const uint2 *>(p);
            } else {
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    c[k].x |= static_cast<uint32_t>(p[z]) << 8 * z, c[k].y |= static_cast<uint32_t>(p[4 + z]) << 8 * z;
            }
            s[k] = scales[page * s_page + (slot >> a.shift) * s_block];
        }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        if (!(good >> k & 1)) continue;
        float x[4], y[4];
        decode4(c[k].x, a.codes, x);
        decode4(c[k].y, a.codes, y);
#pragma unroll
        for (int z = 0; z < 4; ++z) x[z] *= s[k], y[z] *= s[k];
        const int64_t o = (t0 + k * groups + g) * h.yt + head * h.yh + 8 * u;
        if constexpr (WIDE) {
            if (h.ytype == Q4K_F32) {
                float *d = static_cast<float *>(h.y) + o;
                *reinterpret_cast<float4 *>(d) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4 *>(d + 4) = make_float4(y[0], y[1], y[2], y[3]);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(h.y) + o) =
                    make_uint4(attn::pack2(x[0], x[1], h.ytype), attn::pack2(x[2], x[3], h.ytype), attn::pack2(y[0], y[1], h.ytype),
                               attn::pack2(y[2], y[3], h.ytype));
            }
        } else {
#pragma unroll
            for (int z = 0; z < 4; ++z) store1(h.y, h.ytype, o + z, x[z]), store1(h.y, h.ytype, o + 4 + z, y[z]);
        }
    }
}

// ---------------------------------------------------------------- host

static bool good_type(int t) { return t == Q4K_F32 || t == Q4K_F16 || t == Q4K_BF16; }
static int size_of(int t) { return t == Q4K_F32 ? 4 : 2; }
static bool off(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Whether every row of a tensor starts on a 16-byte boundary.
static bool wide_rows(const void *p, int type, int64_t token, int64_t head)
{
    const int64_t per = 16 / size_of(type);
    return !off(p, 16) && token % per == 0 && head % per == 0;
}

static bool wide_codes(const void *p, int64_t page, int64_t slot, int64_t head)
{
    return !off(p, 8) && page % 8 == 0 && slot % 8 == 0 && head % 8 == 0;
}

static bool wide_weight(const float *p, int64_t head) { return !off(p, 16) && head % 4 == 0; }

static cudaError_t launch(void (*kern)(Args), const Args &a, int64_t ctas, int threads, void *stream)
{
    if (ctas < 1 || ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = static_cast<unsigned>(ctas);
    cfg.blockDim = static_cast<unsigned>(threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = a.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// Pairs of a lane, and lanes of a row.
static int pairs_of(int64_t dim, int64_t rot, bool wide) { return wide && dim > 64 && dim % 16 == 0 && rot % 16 == 0 ? 8 : 4; }
static int lanes_of(int64_t dim, int e)
{
    int n = 8;
    while (2 * e * n < dim) n *= 2;
    return n;
}

// Rows a lane group of the queries' side: several where one each would make more
// warps than the GPU holds.
static bool many_rows(int64_t tokens, int heads, int lanes, int sms)
{
    return tokens * heads * lanes / 32 >= 32LL * sms;
}

static bool finite_eps(float e) { return std::isfinite(e) && e >= 0.0f; }

// Sizes of a cache's side of the arguments.
static void fill_cache(Args &p, const q4k_paged_cache8 *c8)
{
    const q4k_paged_cache &c = c8->cache;
    p.at.page_table = c.page_table, p.at.seq_start = c.seq_start, p.at.kv_len = c.kv_len;
    p.at.pages = c.pages, p.at.table_stride = c.page_table_stride, p.at.max_pages = c.max_pages;
    p.at.page_size = static_cast<int>(c.page_size), p.at.batch = static_cast<int>(c.batch), p.at.tokens = static_cast<int>(c.tokens);
    p.kc = static_cast<uint8_t *>(c.k), p.vc = static_cast<uint8_t *>(c.v), p.ks = c8->k_scale, p.vs = c8->v_scale;
    p.k_page = c.k_page_stride, p.k_slot = c.k_slot_stride, p.k_head = c.k_head_stride;
    p.v_page = c.v_page_stride, p.v_slot = c.v_slot_stride, p.v_head = c.v_head_stride;
    p.ks_page = c8->k_scale_page_stride, p.ks_block = c8->k_scale_block_stride, p.ks_head = c8->k_scale_head_stride;
    p.vs_page = c8->v_scale_page_stride, p.vs_block = c8->v_scale_block_stride, p.vs_head = c8->v_scale_head_stride;
    p.dim = static_cast<int>(c.dim), p.codes = c.type, p.block = static_cast<int>(c8->block);
    for (p.shift = 0; (1 << p.shift) < p.block;) ++p.shift;
    p.over_dim = 1.0f / static_cast<float>(p.dim);
}

}  // namespace cache8

q4k_status check_cache8(const q4k_paged_cache8 *c)
{
    using namespace cache8;
    if (!c || (c->cache.type != Q4K_I8 && c->cache.type != Q4K_E4M3)) return Q4K_ERR_INVALID_ARG;
    q4k_paged_cache as16 = c->cache;   // sizes and index pointers are checked alike; codes have no alignment
    as16.type = Q4K_F16;
    const uintptr_t k = reinterpret_cast<uintptr_t>(as16.k), v = reinterpret_cast<uintptr_t>(as16.v);
    as16.k = reinterpret_cast<void *>((k + 1) & ~uintptr_t{1}), as16.v = reinterpret_cast<void *>((v + 1) & ~uintptr_t{1});
    const q4k_status st = check_cache(&as16);
    if (st == Q4K_ERR_INVALID_ARG) return st;
    if (c->cache.dim % 8 || c->cache.dim > kMaxDim || c->block < 1 || c->block > kMaxBlock || (c->block & (c->block - 1)) ||
        c->cache.page_size % c->block)
        return Q4K_ERR_INVALID_ARG;
    if (c->cache.tokens > 0 && c->cache.batch > 0 && (!c->k_scale || !c->v_scale)) return Q4K_ERR_INVALID_ARG;
    return st != Q4K_OK || off(c->k_scale, 4) || off(c->v_scale, 4) ? Q4K_ERR_MISALIGNED : Q4K_OK;
}

q4k_paged_cache8 with_used_strides(q4k_paged_cache8 c)
{
    c.cache = with_used_strides(c.cache);
    const int64_t pages = c.cache.pages, blocks = c.cache.page_size / c.block, heads = c.cache.heads;
    c.k_scale_page_stride = used_stride(c.k_scale_page_stride, pages), c.v_scale_page_stride = used_stride(c.v_scale_page_stride, pages);
    c.k_scale_block_stride = used_stride(c.k_scale_block_stride, blocks);
    c.v_scale_block_stride = used_stride(c.v_scale_block_stride, blocks);
    c.k_scale_head_stride = used_stride(c.k_scale_head_stride, heads), c.v_scale_head_stride = used_stride(c.v_scale_head_stride, heads);
    return c;
}

q4k_status norm_rope_impl(const q4k_norm_rope_args *a, void *stream)
{
    using namespace cache8;
    if (!a || a->tokens < 0 || a->tokens > 0x7FFFFFFF || a->dim < 8 || a->dim > kMaxDim || a->dim % 8 || a->rot < 0 || a->rot % 2 ||
        a->rot > a->dim || a->table_rows < 0 || !finite_eps(a->eps) || (a->interleaved & ~1) || (a->flags & ~Q4K_FLAG_PDL))
        return Q4K_ERR_INVALID_ARG;
    const bool two = a->k.x != nullptr;
    if (two != (a->k.y != nullptr)) return Q4K_ERR_INVALID_ARG;
    bool misaligned = off(a->pos, 4) || off(a->table, 4), wide = a->rot % 8 == 0 && !off(a->table, 16);
    Args p{};
    Heads *to[2] = {&p.q, &p.k};
    const q4k_heads *from[2] = {&a->q, &a->k};
    for (int i = 0; i < (two ? 2 : 1); ++i) {
        const q4k_heads &h = *from[i];
        if (h.heads < 1 || h.heads > 65536 || !good_type(h.x_type) || !good_type(h.y_type)) return Q4K_ERR_INVALID_ARG;
        misaligned = misaligned || off(h.x, size_of(h.x_type)) || off(h.y, size_of(h.y_type)) || off(h.weight, 4);
        *to[i] = Heads{h.x, h.y, h.weight, used_stride(h.x_token_stride, a->tokens), used_stride(h.x_head_stride, h.heads),
                       used_stride(h.y_token_stride, a->tokens), used_stride(h.y_head_stride, h.heads),
                       used_stride(h.weight_head_stride, h.heads), static_cast<int>(h.heads), h.x_type, h.y_type,
                       static_cast<int>(a->rot)};
        const Heads &t = *to[i];
        wide = wide && wide_rows(h.x, h.x_type, t.xt, t.xh) && wide_rows(h.y, h.y_type, t.yt, t.yh) && wide_weight(h.weight, t.wh);
    }
    if (a->tokens > 0 && (!a->q.x || !a->q.y || (a->rot && (!a->pos || !a->table)))) return Q4K_ERR_INVALID_ARG;
    if (misaligned) return Q4K_ERR_MISALIGNED;
    int sms = 0;
    const q4k_status st = check_device(&sms);
    if (st != Q4K_OK || a->tokens == 0) return st;
    p.at.pos = a->pos, p.at.table_rows = a->table_rows, p.at.tokens = static_cast<int>(a->tokens);
    p.table = a->table, p.dim = static_cast<int>(a->dim), p.rot = static_cast<int>(a->rot), p.inter = a->interleaved;
    const int e = pairs_of(a->dim, a->rot, wide);
    p.lanes = lanes_of(a->dim, e), p.over_dim = 1.0f / static_cast<float>(p.dim);
    p.eps = a->eps, p.pdl = a->flags & Q4K_FLAG_PDL;
    const int heads = p.q.heads + p.k.heads;
    const bool many = wide && many_rows(a->tokens, heads, p.lanes, sms);
    const int64_t each = chunk_heads(many ? 16 / e : 1, p.lanes);
    const int64_t warps = a->tokens * ((p.q.heads + each - 1) / each + (p.k.heads + each - 1) / each);
    auto pick = [&](auto inter) {
        constexpr bool INTER = decltype(inter)::value;
        return e == 8 ? (many ? norm_rope_kernel<true, 2, 8, INTER> : norm_rope_kernel<true, 1, 8, INTER>)
                      : (many ? norm_rope_kernel<true, 4, 4, INTER> : norm_rope_kernel<true, 1, 4, INTER>);
    };
    auto kern = !wide ? norm_rope_kernel<false, 1, 4, false> : p.inter ? pick(std::true_type{}) : pick(std::false_type{});
    return launch(kern, p, (warps + kWarps - 1) / kWarps, kWarps * 32, stream) == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA;
}

q4k_status kv_append8_impl(const q4k_paged_cache8 *c8, const q4k_append8_args *a8, void *stream)
{
    using namespace cache8;
    q4k_status st = check_cache8(c8);
    if (st == Q4K_ERR_INVALID_ARG || !a8) return Q4K_ERR_INVALID_ARG;
    const q4k_paged_cache8 used = with_used_strides(*c8);
    const q4k_paged_cache *c = &used.cache;
    const q4k_append_args *a = &a8->a;
    const bool some = c->tokens > 0 && c->batch > 0;
    if (a->rot < 0 || a->rot % 2 || a->rot > c->dim || a->rot > kMaxRot || a->table_rows < 0 || !good_type(a->kv_type) ||
        (a->interleaved & ~1) || (a->flags & ~Q4K_FLAG_PDL) || (a->q == nullptr) != (a->q_out == nullptr) || !finite_eps(a8->eps))
        return Q4K_ERR_INVALID_ARG;
    if (a->q && (a->q_heads < 1 || a->q_heads > 65536 || !good_type(a->q_type) || !good_type(a->q_out_type))) return Q4K_ERR_INVALID_ARG;
    if (some && (!a->k || !a->v || (a->rot && !a->table))) return Q4K_ERR_INVALID_ARG;
    // slots or scales that are one and the same would take what was written last
    auto same = [](int64_t stride, int64_t n) { return n > 1 && stride == 0; };
    const int64_t blocks = c->page_size / used.block;
    if (same(c->k_page_stride, c->pages) || same(c->k_slot_stride, c->page_size) || same(c->k_head_stride, c->heads) ||
        same(c->v_page_stride, c->pages) || same(c->v_slot_stride, c->page_size) || same(c->v_head_stride, c->heads) ||
        same(used.k_scale_page_stride, c->pages) || same(used.k_scale_block_stride, blocks) || same(used.k_scale_head_stride, c->heads) ||
        same(used.v_scale_page_stride, c->pages) || same(used.v_scale_block_stride, blocks) || same(used.v_scale_head_stride, c->heads))
        return Q4K_ERR_INVALID_ARG;
    if (st != Q4K_OK) return st;
    if (off(a->k, size_of(a->kv_type)) || off(a->v, size_of(a->kv_type)) || off(a->pos, 4) || off(a->table, 4) ||
        off(a8->q_weight, 4) || off(a8->k_weight, 4) ||
        (a->q && (off(a->q, size_of(a->q_type)) || off(a->q_out, size_of(a->q_out_type)))))
        return Q4K_ERR_MISALIGNED;
    int sms = 0;
    st = check_device(&sms);
    if (st != Q4K_OK || !some) return st;
    Args p{};
    fill_cache(p, &used);
    const int heads = static_cast<int>(c->heads), rot = static_cast<int>(a->rot);
    const int64_t n = c->tokens;
    p.k = Heads{a->k, nullptr, a8->k_weight, used_stride(a->k_token_stride, n), used_stride(a->k_head_stride, heads), 0, 0,
                used_stride(a8->k_weight_head_stride, heads), heads, a->kv_type, 0, rot};
    p.v = Heads{a->v, nullptr, nullptr, used_stride(a->v_token_stride, n), used_stride(a->v_head_stride, heads), 0, 0, 0, heads,
                a->kv_type, 0, 0};
    bool wide = rot % 8 == 0 && !off(a->table, 16) && wide_rows(a->k, a->kv_type, p.k.xt, p.k.xh) &&
                wide_rows(a->v, a->kv_type, p.v.xt, p.v.xh) && wide_codes(c->k, p.k_page, p.k_slot, p.k_head) &&
                wide_codes(c->v, p.v_page, p.v_slot, p.v_head) && wide_weight(a8->k_weight, p.k.wh);
    if (a->q) {
        p.q = Heads{a->q, a->q_out, a8->q_weight, used_stride(a->q_token_stride, n), used_stride(a->q_head_stride, a->q_heads),
                    used_stride(a->q_out_token_stride, n), used_stride(a->q_out_head_stride, a->q_heads),
                    used_stride(a8->q_weight_head_stride, a->q_heads), static_cast<int>(a->q_heads), a->q_type, a->q_out_type, rot};
        wide = wide && wide_rows(a->q, a->q_type, p.q.xt, p.q.xh) && wide_rows(a->q_out, a->q_out_type, p.q.yt, p.q.yh) &&
               wide_weight(a8->q_weight, p.q.wh);
    }
    p.at.pos = a->pos, p.at.table_rows = a->table_rows;
    p.table = a->table, p.rot = rot, p.inter = a->interleaved, p.eps = a8->eps, p.pdl = a->flags & Q4K_FLAG_PDL;
    const int e = pairs_of(c->dim, rot, wide);
    p.lanes = lanes_of(c->dim, e);
    const int groups = 32 / p.lanes, hold = rows_of(e) * groups;
    p.run = std::max(p.block, hold), p.warps = p.run / hold;
    const int64_t slots = 2 * static_cast<int64_t>(p.at.batch) + n / p.run + 1;
    if (slots > 0x7FFFFFFF) return Q4K_ERR_INVALID_ARG;
    p.slots = static_cast<int>(slots);
    const int warps = std::max(kWarps, p.warps), per = warps / p.warps;
    const int64_t kv_ctas = (slots * 2 * heads + per - 1) / per;
    const bool many = wide && many_rows(n, p.q.heads, p.lanes, sms);
    const int64_t each = chunk_heads(many ? 16 / e : 1, p.lanes), q_warps = n * ((p.q.heads + each - 1) / each);
    if (kv_ctas + q_warps > 0x7FFFFFFF) return Q4K_ERR_INVALID_ARG;
    p.kv_ctas = static_cast<int>(kv_ctas);
    // Many waves of CTAs gain by a fifth on each SM what the spilled registers cost: 7000 tokens of 32 / 8 bf16 heads,
    // normed, 59.3 us (four CTAs 63.2), of 28 / 4 fp32 heads 54.9 (57.0); 2048 tokens 18.5 (18.6); 1500 fp32 tokens,
    // three waves, 17.7 (14.5).
    const int64_t ctas = kv_ctas + (q_warps + warps - 1) / warps;
    const bool five = ctas * warps >= 24LL * kWarps * sms;
    auto pick = [&](auto inter) {
        constexpr bool INTER = decltype(inter)::value;
        return e == 8 ? (!many  ? append8_kernel<true, 1, 8, INTER, false>
                         : five ? append8_kernel<true, 2, 8, INTER, true>
                                : append8_kernel<true, 2, 8, INTER, false>)
                      : (many ? append8_kernel<true, 4, 4, INTER, false> : append8_kernel<true, 1, 4, INTER, false>);
    };
    auto kern = !wide ? append8_kernel<false, 1, 4, false, false> : p.inter ? pick(std::true_type{}) : pick(std::false_type{});
    return launch(kern, p, ctas, warps * 32, stream) == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA;
}

q4k_status kv_read8_impl(const q4k_paged_cache8 *c8, const q4k_read8_args *a, void *stream)
{
    using namespace cache8;
    q4k_status st = check_cache8(c8);
    if (st == Q4K_ERR_INVALID_ARG || !a || !good_type(a->type) || (a->flags & ~Q4K_FLAG_PDL)) return Q4K_ERR_INVALID_ARG;
    const q4k_paged_cache8 used = with_used_strides(*c8);
    const q4k_paged_cache *c = &used.cache;
    if (st != Q4K_OK) return st;
    if (off(a->k, size_of(a->type)) || off(a->v, size_of(a->type))) return Q4K_ERR_MISALIGNED;
    st = check_device(nullptr);
    if (st != Q4K_OK || c->tokens == 0 || c->batch == 0 || (!a->k && !a->v)) return st;
    Args p{};
    fill_cache(p, &used);
    const int heads = static_cast<int>(c->heads);
    const int64_t n = c->tokens;
    p.k.y = a->k, p.k.yt = used_stride(a->k_token_stride, n), p.k.yh = used_stride(a->k_head_stride, heads), p.k.ytype = a->type;
    p.v.y = a->v, p.v.yt = used_stride(a->v_token_stride, n), p.v.yh = used_stride(a->v_head_stride, heads), p.v.ytype = a->type;
    p.k.heads = a->k ? heads : 0, p.v.heads = a->v ? heads : 0;
    p.pdl = a->flags & Q4K_FLAG_PDL;
    const bool wide = wide_codes(c->k, p.k_page, p.k_slot, p.k_head) && wide_codes(c->v, p.v_page, p.v_slot, p.v_head) &&
                      wide_rows(a->k, a->type, p.k.yt, p.k.yh) && wide_rows(a->v, a->type, p.v.yt, p.v.yh);
    p.lanes = lanes_of(c->dim, 4);   // 8 codes a lane
    const int hold = 8 * (32 / p.lanes);
    const int64_t warps = (n + hold - 1) / hold * (p.k.heads + p.v.heads);
    auto kern = wide ? read8_kernel<true> : read8_kernel<false>;
    return launch(kern, p, (warps + kWarps - 1) / kWarps, kWarps * 32, stream) == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA;
}

}  // namespace q4k
