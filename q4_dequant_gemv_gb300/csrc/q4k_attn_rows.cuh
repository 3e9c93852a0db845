// q4k_attn_rows.cuh -- attention of a few query rows per cache head (decode and
// verification) on mma.sync, keys and values straight from global memory into
// registers.
//
// Such a call reads every visible key and value once for 1 to 16 query rows: at
// 7 rows 7 flops a byte, far below what any tensor path offers, so the kernel is
// bound by memory and by how many loads are in flight.  A warp takes 16 keys at
// a time and needs no barrier and no shared memory for them:
//   S^T = K Q^T: A fragment = 16 keys x 16 d.  The order of d inside the
//     contraction is free, so a thread's fragment registers for two MMAs are one
//     16-byte load of 8 consecutive d of its key; Q is laid out to match.
//   O^T = V^T P^T: A fragment = 16 d x 16 keys.  The order of d in the rows is
//     free too: a thread loads 8 consecutive d of four keys (16 bytes each) and
//     pairs the keys with byte permutes, which gives the fragments of four MMAs.
//     P^T comes from the S^T accumulators by an 8x8 transpose (movmatrix).
// The queries are the 8-wide N side, so 7 or 8 heads of a group fill it.
// Softmax runs per warp over its own keys (running maximum, sum and O rescaled
// when the maximum grows); the warps of a CTA join once per tile.
//
// Parts: with fp32 queries or outputs, Q and P enter as PARTS 16-bit parts (3
// bf16 or 2 fp16: 24 and 22 bits), each an MMA of its own; the products are
// exact in fp32.  fp16: a power of two per query row brings max|q| to 2^14, and
// P carries 2^14, so the low parts stay above fp16's subnormals.
#pragma once
#include <cuda_runtime.h>

#include "q4k_attn.cuh"
#include "ptx.cuh"

namespace q4k {
namespace attn {

constexpr int kRowsWarps = 8;
constexpr int kRowsThreads = kRowsWarps * 32;
constexpr int kRowsUnit = 16 * kRowsWarps;   // keys per unit

template <int CT>
__device__ __forceinline__ void mma_t(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1)
{
    if constexpr (CT == Q4K_F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint4 load_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// x as PARTS packed pairs; each part takes what the earlier ones left.
template <int CT, int PARTS>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[PARTS])
{
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        p[i] = pack2(x, y, CT);
        if (i + 1 < PARTS) {
            const float2 r = unpack2(p[i], CT);
            x -= r.x, y -= r.y;
        }
    }
}

template <int CT, int PARTS, int NT, int DP>
struct RowsShared {
    static constexpr int R = 8 * NT;
    using Plan = Split<R, kRowsUnit, kRowsThreads, 16>;
    typename Plan::Shared plan;
    uint4 q[PARTS][NT][DP / 32][32];       // B fragments of Q, lane-major
    float red[kRowsWarps][8][DP];          // O of the warps, one n8 tile at a time
    float m[kRowsWarps][R], l[kRowsWarps][R];
    float scale[R], slope[R];
    int lo[R], hi[R], pos[R];              // visible keys and position of each row (position relative to `pos0`)
    float wm[R], wl[R];                    // joined statistics
    unsigned int arrived;
};

template <int CT, int PARTS, int NT, int DP>
__global__ void __launch_bounds__(kRowsThreads, (NT == 1 && DP <= 128) ? 2 : 1) rows_kernel(const Args a)
{
    using Sh = RowsShared<CT, PARTS, NT, DP>;
    constexpr int R = Sh::R, CH = DP / 32, VH = DP / 64;
    constexpr float kShift = CT == Q4K_F16 ? 14.0f : 0.0f;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Sh &sh = *reinterpret_cast<Sh *>(smem_raw);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;

    typename Sh::Plan plan(a, sh.plan);
    const int64_t total = static_cast<int64_t>(plan.per_head) * a.kv_heads;
    if (total == 0) return;
    const int n = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
    const int cta = blockIdx.x;
    if (cta >= n) return;
    int64_t u = share_begin(total, n, cta);
    const int64_t u_end = share_begin(total, n, cta + 1);

    const uint16_t *kbase = static_cast<const uint16_t *>(a.k), *vbase = static_cast<const uint16_t *>(a.v);
    const int psize = static_cast<int>(a.page_size);

    while (u < u_end) {
        const int head = static_cast<int>(u / plan.per_head);
        int off;
        const Tile t = plan.locate(static_cast<uint32_t>(u - static_cast<int64_t>(head) * plan.per_head), off);
        const int64_t u0 = u - off;
        const int todo = static_cast<int>(min(static_cast<int64_t>(t.units - off), u_end - u));

        // ---- the tile's rows: scale, visible range, fragments of Q
        __syncthreads();   // the previous tile's shared data is done with
        for (int r = w; r < R; r += kRowsWarps) {   // a warp per row
            const bool live = r < t.rows;
            const int row = t.first + r, tok = row / a.group, hq = head * a.group + row % a.group;
            float x[DP / 32];
            float mx = 0.0f;
            const int64_t base = (t.tok0 + tok) * a.q_token + hq * a.q_head;
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                const int d = 32 * c + lane;
                x[c] = 0.0f;
                if (live && d < a.dim) {
                    if (a.q_type == Q4K_F32) x[c] = static_cast<const float *>(a.q)[base + d];
                    else if (a.q_type == Q4K_F16) x[c] = __half2float(static_cast<const __half *>(a.q)[base + d]);
                    else x[c] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[base + d]);
                }
                mx = fmaxf(mx, fabsf(x[c]));
            }
            int e = 0;
            if (PARTS > 1 && CT == Q4K_F16) {   // max|q| to [2^14, 2^15)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const uint32_t b = __float_as_uint(mx);
                const int ex = static_cast<int>(b >> 23);
                if (b != 0u && ex != 255) e = max(-126, min(126, 141 - ex));
            }
            const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                // element d = 32c + 8j + i of the row: half i & 1 of word i >> 1 of lane 4 (r % 8) + j
                float v = x[c] * up;
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    const uint32_t h = pack2(v, 0.0f, CT);
                    reinterpret_cast<uint16_t *>(&sh.q[p][r >> 3][c][4 * (r & 7) + (lane >> 3)])[lane & 7] =
                        static_cast<uint16_t>(h & 0xFFFFu);
                    v -= unpack2(h, CT).x;
                }
            }
            if (lane == 0) {
                Range v{0, 0};
                if (live) v = token_range(a, t.seq, t.pos0 + tok, t.tok0 + tok, t.len);
                sh.lo[r] = static_cast<int>(v.lo), sh.hi[r] = static_cast<int>(v.hi);
                sh.pos[r] = tok;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                sh.scale[r] = (a.softcap > 0.0f ? a.scale / a.softcap : a.scale * kLog2e) * down;
                sh.slope[r] = live && a.slopes ? a.slopes[hq] * kLog2e : 0.0f;
            }
        }
        __syncthreads();

        float scl[NT][2], slope[NT][2];
        int lo[NT][2], hi[NT][2], ptok[NT][2];
        int in_lo = 0, in_hi = 0x7FFFFFFF;   // keys that every live row sees
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 8 * nt + 2 * t4 + j;
                scl[nt][j] = sh.scale[r], slope[nt][j] = sh.slope[r];
                lo[nt][j] = sh.lo[r], hi[nt][j] = sh.hi[r], ptok[nt][j] = sh.pos[r];
            }
        for (int r = 0; r < t.rows; ++r) in_lo = max(in_lo, sh.lo[r]), in_hi = min(in_hi, sh.hi[r]);

        float m[NT][2], l[NT][2], o[NT][2 * CH][4];   // o[..][4 h + i]: d = 64 h + 8 g + 2 i (+1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) m[nt][j] = -INFINITY, l[nt][j] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * CH; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
        }

        // ---- the keys: 16 per warp and step
        const int32_t *pages = a.page_table + static_cast<int64_t>(t.seq) * a.table_stride;
        const int kb0 = t.lo + off * kRowsUnit + 16 * w;
        uint4 kf[2][CH], vf[4][VH];
        // page and slot of this lane's key (key kb + lane % 16)
        auto place = [&](int kb, int &pg, int &slot) {
            const int key = kb + (lane & 15);
            pg = 0, slot = 0;
            if (key < t.from || key >= t.hi) return;
            const int e = key / psize;
            slot = key - e * psize;
            pg = pages[e];
            if (pg < 0 || pg >= a.pages) {
                atomicOr(a.error, 4u);
                pg = 0;
            }
        };
        auto load_k = [&](int kb, int pg, int slot) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r;
                const int p = __shfl_sync(0xffffffffu, pg, row), sl = __shfl_sync(0xffffffffu, slot, row);
                const uint16_t *s = kbase + p * a.k_page + sl * a.k_slot + head * a.k_head + 8 * t4;
                const bool live = kb + row >= t.from && kb + row < t.hi;
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    kf[r][c] = live && 32 * c + 8 * t4 < a.dim ? load_stream(s + 32 * c) : make_uint4(0, 0, 0, 0);
            }
        };
        auto load_v = [&](int kb, int pg, int slot) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 2 * t4 + (r & 1) + 8 * (r >> 1);
                const int p = __shfl_sync(0xffffffffu, pg, row), sl = __shfl_sync(0xffffffffu, slot, row);
                const uint16_t *s = vbase + p * a.v_page + sl * a.v_slot + head * a.v_head + 8 * g;
                const bool live = kb + row >= t.from && kb + row < t.hi;
#pragma unroll
                for (int h = 0; h < VH; ++h)
                    vf[r][h] = live && 64 * h + 8 * g < a.dim ? load_stream(s + 64 * h) : make_uint4(0, 0, 0, 0);
            }
        };

        int pg, slot;
        place(kb0, pg, slot);
        if (kb0 < t.hi) load_k(kb0, pg, slot), load_v(kb0, pg, slot);
        for (int i = 0; i < todo; ++i) {
            const int kb = kb0 + i * kRowsUnit;
            if (kb >= t.hi) break;
            const int kn = kb + kRowsUnit;
            const bool more = i + 1 < todo && kn < t.hi;
            if (more) place(kn, pg, slot);

            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // chains of their own: the two k-steps of a load (one part), or the parts
                constexpr int CHAINS = PARTS > 1 ? PARTS : 2;
                float acc[CHAINS][4] = {};
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        const uint4 b = sh.q[p][nt][c][lane];
                        mma_t<CT>(acc[p], kf[0][c].x, kf[1][c].x, kf[0][c].y, kf[1][c].y, b.x, b.y);
                        mma_t<CT>(acc[PARTS > 1 ? p : 1], kf[0][c].z, kf[1][c].z, kf[0][c].w, kf[1][c].w, b.z, b.w);
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (PARTS > 1) {
                        // an infinite key: the first part has its sign, the others may be 0 or of the other sign
                        float rest = acc[PARTS - 1][j];
#pragma unroll
                        for (int p = PARTS - 2; p > 0; --p) rest += acc[p][j];
                        const bool finite = fabsf(acc[0][j]) < INFINITY;
                        s[nt][j] = finite ? acc[0][j] + rest : acc[0][j];
                    } else {
                        s[nt][j] = acc[0][j] + acc[1][j];
                    }
                }
            }
            if (more) load_k(kn, pg, slot);

            const bool all = kb >= in_lo && kb + 16 <= in_hi;
            uint32_t pb[NT][PARTS][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x = s[nt][j] * scl[nt][j & 1];
                    if (a.softcap > 0.0f) {
                        const float th = PARTS > 1 ? tanhf(x) : 1.0f - 2.0f * rcp(ex2(2.0f * kLog2e * x) + 1.0f);
                        x = a.softcap * kLog2e * th;
                    }
                    const int key = kb + g + 8 * (j >> 1);
                    if (a.slopes)
                        x -= slope[nt][j & 1] *
                             fabsf(static_cast<float>(t.pos0 + ptok[nt][j & 1] - key));
                    if (!all && (key < lo[nt][j & 1] || key >= hi[nt][j & 1])) x = -INFINITY;
                    s[nt][j] = x;
                }
                float mx[2], f[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v = fmaxf(s[nt][j], s[nt][j + 2]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    mx[j] = fmaxf(m[nt][j], v);
                    f[j] = mx[j] == -INFINITY ? 1.0f : ex2(m[nt][j] - mx[j]);
                    m[nt][j] = mx[j];
                    l[nt][j] *= f[j];
                }
                if (__any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
                    for (int q = 0; q < 2 * CH; ++q) {
                        o[nt][q][0] *= f[0], o[nt][q][1] *= f[1];
                        o[nt][q][2] *= f[0], o[nt][q][3] *= f[1];
                    }
                }
                float e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float base = mx[j & 1] == -INFINITY ? 0.0f : mx[j & 1] - kShift;
                    e[j] = ex2(s[nt][j] - base);
                    l[nt][j & 1] += e[j];
                }
                uint32_t p0[PARTS], p1[PARTS];
                split2<CT, PARTS>(e[0], e[1], p0);
                split2<CT, PARTS>(e[2], e[3], p1);
#pragma unroll
                for (int p = 0; p < PARTS; ++p) pb[nt][p][0] = transpose8(p0[p]), pb[nt][p][1] = transpose8(p1[p]);
            }
#pragma unroll
            for (int h = 0; h < VH; ++h) {
                const uint32_t *v0 = &vf[0][h].x, *v1 = &vf[1][h].x, *v2 = &vf[2][h].x, *v3 = &vf[3][h].x;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t a0 = __byte_perm(v0[q], v1[q], 0x5410), a1 = __byte_perm(v0[q], v1[q], 0x7632);
                    const uint32_t a2 = __byte_perm(v2[q], v3[q], 0x5410), a3 = __byte_perm(v2[q], v3[q], 0x7632);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int p = PARTS - 1; p >= 0; --p)
                            mma_t<CT>(o[nt][4 * h + q], a0, a1, a2, a3, pb[nt][p][0], pb[nt][p][1]);
                }
            }
            if (more) load_v(kn, pg, slot);
        }

        // ---- join the warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
                if (g == 0) sh.m[w][8 * nt + 2 * t4 + j] = m[nt][j], sh.l[w][8 * nt + 2 * t4 + j] = l[nt][j];
            }
        __syncthreads();
        if (tid < R) {
            float mx = -INFINITY, ls = 0.0f;
            for (int i = 0; i < kRowsWarps; ++i) mx = fmaxf(mx, sh.m[i][tid]);
            for (int i = 0; i < kRowsWarps; ++i)
                ls += sh.l[i][tid] * weight(sh.m[i][tid], mx);
            sh.wm[tid] = mx, sh.wl[tid] = ls;
        }
        const bool split = todo < t.units;
        const int64_t pslot = 2 * static_cast<int64_t>(cta) + (off == 0 ? 1 : 0);
        float *part = a.part + pslot * (R * (DP + 2));
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int q = 2 * t4 + j;
                const float mx = sh.wm[8 * nt + q];
                const float f = weight(m[nt][j], mx);
#pragma unroll
                for (int h = 0; h < VH; ++h) {
                    float4 *dst = reinterpret_cast<float4 *>(&sh.red[w][q][64 * h + 8 * g]);
                    dst[0] = make_float4(o[nt][4 * h][j] * f, o[nt][4 * h][j + 2] * f, o[nt][4 * h + 1][j] * f,
                                         o[nt][4 * h + 1][j + 2] * f);
                    dst[1] = make_float4(o[nt][4 * h + 2][j] * f, o[nt][4 * h + 2][j + 2] * f,
                                         o[nt][4 * h + 3][j] * f, o[nt][4 * h + 3][j + 2] * f);
                }
            }
            __syncthreads();
            for (int i = tid; i < 8 * DP / 4; i += kRowsThreads) {
                const int q = i / (DP / 4), d = 4 * (i % (DP / 4)), r = 8 * nt + q;
                float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kRowsWarps; ++k) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sh.red[k][q][d]);
                    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                }
                if (r < t.rows && d < a.dim) {
                    if (split) {
                        *reinterpret_cast<float4 *>(part + r * DP + d) = v;
                    } else {
                        const float ls = sh.wl[r], inv = ls == 0.0f ? 0.0f : 1.0f / ls;
                        const int row = t.first + r;
                        const int64_t at = (t.tok0 + row / a.group) * a.out_token +
                                           (head * a.group + row % a.group) * a.out_head + d;
                        store4(a.out, a.out_type, at, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                    }
                }
            }
            __syncthreads();
        }
        if (tid < t.rows) {
            if (split) {
                part[R * DP + tid] = sh.wm[tid], part[R * DP + R + tid] = sh.wl[tid];
            } else if (a.lse) {
                const int row = t.first + tid;
                const float ls = sh.wl[tid];
                a.lse[static_cast<int64_t>(t.tok0 + row / a.group) * a.heads + head * a.group + row % a.group] =
                    ls == 0.0f ? -INFINITY : (sh.wm[tid] + log2f(ls) - kShift) * kLn2;
            }
        }

        // ---- a split tile: the last CTA to arrive adds the parts in key order
        if (split) {
            const int c0 = share_owner(total, n, u0), c1 = share_owner(total, n, u0 + t.units - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0) sh.arrived = atomicAdd(a.ticket + c0, 1u);
            __syncthreads();
            if (sh.arrived == static_cast<unsigned int>(c1 - c0)) {
                __threadfence();
                auto slot_of = [&](int c) { return a.part + (2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * (R * (DP + 2)); };
                for (int i = tid; i < R * DP / 4; i += kRowsThreads) {
                    const int r = i / (DP / 4), d = 4 * (i % (DP / 4));
                    if (r >= t.rows || d >= a.dim) continue;
                    float mx = -INFINITY;
                    for (int c = c0; c <= c1; ++c) mx = fmaxf(mx, __ldcg(slot_of(c) + R * DP + r));
                    float4 v = make_float4(0, 0, 0, 0);
                    float ls = 0.0f;
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c) {
                        const float *p = slot_of(c);
                        const float pm = __ldcg(p + R * DP + r);
                        const float f = weight(pm, mx);
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(p + r * DP + d));
                        ls += f * __ldcg(p + R * DP + R + r);
                        v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
                    }
                    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
                    const int row = t.first + r;
                    const int64_t tok = t.tok0 + row / a.group;
                    const int hq = head * a.group + row % a.group;
                    store4(a.out, a.out_type, tok * a.out_token + hq * a.out_head + d,
                           make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                    if (a.lse && d == 0)
                        a.lse[tok * a.heads + hq] = ls == 0.0f ? -INFINITY : (mx + log2f(ls) - kShift) * kLn2;
                }
            }
        }
        u += todo;
    }
}

// Launches the kernel of one cache type (in a translation unit of its own).
struct RowsLaunch {
    Args args;
    int sms, parts_many;   // parts_many: fp32 queries or outputs
    cudaStream_t stream;
};
cudaError_t launch_rows_f16(const RowsLaunch &l);
cudaError_t launch_rows_bf16(const RowsLaunch &l);

}  // namespace attn
}  // namespace q4k
