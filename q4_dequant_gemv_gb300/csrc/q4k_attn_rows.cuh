// q4k_attn_rows.cuh -- attention of a few query rows per cache head (decode and
// verification) on mma.sync.
//
// Such a call reads every visible key and value once for 1 to 32 query rows: at
// 7 rows 7 flops a byte, far below what any tensor path offers, so the kernel is
// bound by memory and by how many bytes are in flight.  A warp owns blocks of 16
// keys and a ring of its own in shared memory, fills a slot ahead of time and
// refills it when it has read it: no barrier between warps until they join at
// the end of a tile, and 130 to 190 KB in flight per SM.  Tiles of 32
// rows give each block to two warps, half of the rows each (registers).
//   S^T = K Q^T: A = 16 keys x 16 d (ldmatrix), B = Q^T from shared memory;
//   O^T = V^T P^T: A = 16 d x 16 keys (ldmatrix.trans), B = P^T from the S^T
//   accumulators by an 8x8 transpose (movmatrix).
// The queries are the 8-wide N side, so 7 or 8 heads of a group fill it.
// Softmax runs per warp over its own keys (running maximum, sum and O rescaled
// when the maximum grows).
//
// Slots are filled by TMA boxes of 16 keys x 64 d (128-byte swizzle) where pages
// hold a multiple of 16 keys, else by 16-byte asynchronous copies row by row in
// the same layout.  Rows of V that no row of the tile sees are zero (they may
// hold NaN in memory, and P = 0 would not remove it); such keys' scores are
// replaced.
//
// Parts: with fp32 queries or outputs, Q and P enter as PARTS 16-bit parts (3
// bf16 or 2 fp16: 24 and 22 bits), each an MMA of its own; the products are
// exact in fp32.  fp16: a power of two per query row brings max|q| to 2^14, and
// P carries 2^14, so the low parts stay above fp16's subnormals.
//
// Measured (device): one token of 32 / 8 bf16 heads over 131072 positions 90 us,
// 5.9 TB/s = 89 % of a copy's rate (keys straight into registers 142, rings 97, the
// join in three trips 94); sixteen fp32 tokens of 28 / 4 heads over 4096 26.4 us (58
// without rings, 37 without clusters); one over 1000 7.4 us, five dependent trips to
// memory; four times five tokens over 2000, scores capped, 15.4 us.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "q4k_attn.cuh"
#include "ptx.cuh"

namespace q4k {
namespace attn {

constexpr int kMaxCluster = 8;               // (the portable size)
constexpr int kBlock = 16;                   // keys of a ring slot

// A tile's shape: NT n8 tiles of query rows per warp, RG warps side by side on a
// block of keys, KG such groups; slots of a group's ring (128 to 192 KB in all,
// what the queries and the join leave).
template <int NT, int RG, int DP>
struct RowsShape {
    static constexpr int R = 8 * NT * RG;
    static constexpr int kWarps = DP == 256 ? 4 : 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int KG = kWarps / RG;
    static constexpr int kUnit = kBlock * KG;              // keys per unit
    static constexpr int kSide = kBlock * DP * 2;          // bytes of K (or V) in a slot
    static constexpr int kSlots = RG == 2 ? (DP == 64 ? 8 : 4) : DP == 64 ? 5 : NT * DP >= 512 ? 2 : 3;
};

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

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void st_shared_cluster_v4(uint32_t addr, float4 v)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

__device__ __forceinline__ void st_shared_cluster_v2(uint32_t addr, float x, float y)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// 16 bytes global -> shared, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// One arrival on an mbarrier when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

// tanh within a few ulp: its series where |x| < 0.4 (the next term is 6e-8 of the
// sum there), else 1 - 2 / (e^2|x| + 1).
__device__ __forceinline__ float tanh_close(float x)
{
    const float y = x * x;
    float p = fmaf(y, -8.8632355e-3f, 2.1869488e-2f);
    p = fmaf(p, y, -5.3968254e-2f);
    p = fmaf(p, y, 1.3333333e-1f);
    p = fmaf(p, y, -3.3333333e-1f);
    p = fmaf(p * y, x, x);
    const float e = ex2(2.0f * kLog2e * fabsf(x));
    const float q = copysignf(fmaf(-2.0f, rcp(e + 1.0f), 1.0f), x);
    return fabsf(x) < 0.4f ? p : q;
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

// P carries 2^shift (see above).
template <int CT>
constexpr float rows_shift()
{
    return CT == Q4K_F16 ? 14.0f : 0.0f;
}

template <int CT, int PARTS, int NT, int RG, int DP>
struct RowsShared {
    using Sp = RowsShape<NT, RG, DP>;
    static constexpr int R = Sp::R;
    static constexpr int kRed = DP + 4;    // floats of a row of O when the warps join (no bank conflicts)
    // a group's ring; when the warps join it holds the group's O instead
    static constexpr int kSlotBytes = Sp::kSlots * 2 * Sp::kSide, kOBytes = (R * kRed * 4 + 1023) / 1024 * 1024;
    static constexpr int kRing = kSlotBytes > kOBytes ? kSlotBytes : kOBytes;
    uint8_t ring[Sp::KG][kRing];
    SplitShared<Sp::kThreads> plan;
    uint4 q[PARTS][R / 8][DP / 32][32];    // B fragments of Q, lane-major
    float m[Sp::KG][R], l[Sp::KG][R];
    float scale[R], slope[R];
    int lo[R], hi[R], pos[R];              // visible keys of each row, its token
    // what the ranks of a cluster send: their O for this rank's columns ([rank][row][column
    // quad], whatever the number of ranks), and their statistics
    float4 sent[R * (DP / 4 + kMaxCluster)];
    float2 stat[kMaxCluster][R];
    unsigned long long full[Sp::KG][Sp::kSlots], empty[Sp::KG][Sp::kSlots];
};

// TMA: slots filled by tensor copies (maps), else by cp.async.  DOCS: causal calls
// with kv_start, whose tiles may have holes (an instance of its own: the code for
// them, rarely run, cost calls without them 0.3 to 1 us where it was in one kernel).
template <int CT, int PARTS, int NT, int RG, int DP, bool TMA, bool DOCS>
__global__ void __launch_bounds__(RowsShape<NT, RG, DP>::kThreads, 1) rows_kernel(const __grid_constant__ CacheMaps maps, const Args a)
{
    using Sh = RowsShared<CT, PARTS, NT, RG, DP>;
    using Sp = RowsShape<NT, RG, DP>;
    constexpr int R = Sh::R, ND = DP / 64, KS = DP / 16, WARPS = Sp::kWarps, THREADS = Sp::kThreads, SLOTS = Sp::kSlots;
    constexpr int KG = Sp::KG;
    constexpr int kHalf = kBlock * 128;      // bytes of 16 rows of 64 elements
    constexpr float kShift = rows_shift<CT>();
    extern __shared__ uint8_t smem_raw[];
    Sh &sh = *reinterpret_cast<Sh *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int kg = w % KG, rg = w / KG;      // group of keys, half of the rows

    if (tid < KG * SLOTS) {
        mbar_init(smem_u32(&sh.full[0][0] + tid), TMA ? 1 : 32);
        mbar_init(smem_u32(&sh.empty[0][0] + tid), RG);
        fence_barrier_init();
        if (TMA && tid == 0) prefetch_tensormap(&maps.k), prefetch_tensormap(&maps.v);
    }
    if (a.cluster > 1) cluster_arrive_relaxed();   // (waited for before the first store to another CTA)
    pdl_launch_dependents();
    pdl_wait();                                    // (everything below may come from the kernel before)
    Split<Sp::kUnit, THREADS, kBlock, DOCS> plan(a, sh.plan, R);         // synchronises the CTA
    const int cta = blockIdx.x;
    int64_t total = 0, u = 0, u_end = 1;
    int n = 0;
    bool known = false;   // the first tile has been handed out
    if (!a.cluster) {
        plan.scan();
        total = static_cast<int64_t>(plan.per_head) * a.kv_heads;
        n = sharers(total, gridDim.x);
        if (tid == 0) a.joint[cta].rows = 0;
        if (cta < n) u = share_begin(total, n, cta), u_end = share_begin(total, n, cta + 1);
        else u_end = 0;
        const uint32_t at = per_head_rest(u, plan.per_head);
        known = plan.hand_out(at) && u < u_end;
    }

    const uint32_t ring = smem_u32(sh.ring[kg]);
    // ldmatrix addresses within a slot: row of the lane, chunk before the swizzle
    const int krow = (lane & 7) + 8 * ((lane >> 3) & 1), kch = lane >> 4;
    const int vrow = (lane & 7) + 8 * (lane >> 4), vch = (lane >> 3) & 1;
    uint32_t fills = 0;                      // slots filled so far in this group's ring
    uint32_t reads = 0;                      // phases of the slots' `empty` barriers, a bit each
    bool good = true;                        // no wait has timed out

    while (u < u_end) {
        int head, off, todo;
        int64_t u0 = 0;
        Tile t;
        if (a.cluster) {
            // a cluster per tile and cache head, equal shares of its units
            const int item = cta / a.cluster, rank = cta - item * a.cluster;
            t = plan.template tile<true>(item / a.kv_heads);
            if (!t.rows) {
                if (a.cluster > 1) cluster_wait_acquire();
                return;
            }
            head = item % a.kv_heads;
            off = t.units * rank / a.cluster;
            todo = t.units * (rank + 1) / a.cluster - off;
        } else {
            head = static_cast<int>(quotient(u, plan.per_head));
            if (known) t = sh.plan.first, off = sh.plan.offset;
            else t = plan.locate(static_cast<uint32_t>(u - static_cast<int64_t>(head) * plan.per_head), off);
            known = false;
            u0 = u - off;
            todo = static_cast<int>(min(static_cast<int64_t>(t.units - off), u_end - u));
        }

        const bool holes = DOCS && (t.seq & kHoles);
        if (DOCS) t.seq &= ~kHoles;
        // ---- this group's blocks: key kb0 + i * kUnit, i < count
        const int32_t *pages = a.page_table + static_cast<int64_t>(t.seq) * a.table_stride;
        const int kb0 = t.lo + off * Sp::kUnit + kBlock * kg;
        const int count = good && kb0 < t.hi ? min(todo, (t.hi - kb0 + Sp::kUnit - 1) / Sp::kUnit) : 0;
        // pages and slots of the next 32 blocks, a lane each (TMA): loaded, then checked
        int ids = 0, slots = 0;
        auto look = [&](int first) {
            const int i = first + lane;
            ids = slots = 0;
            if (i < count) {
                int e;
                page_of(a, kb0 + i * Sp::kUnit, e, slots);
                ids = pages[e];
            }
        };
        auto check = [&]() {
            if (ids < 0 || ids >= a.pages) {
                if (!holes) atomicOr(a.error, 4u);
                ids = holes ? -1 : 0;   // (-1: `fill` looks whether any row sees the block)
            }
        };
        // block i into its slot, by the group's first warp
        auto fill = [&](int i, uint32_t f) {
            const int s = static_cast<int>(f % SLOTS);
            const uint32_t dst = ring + s * 2 * Sp::kSide, bar = smem_u32(&sh.full[kg][s]);
            if constexpr (TMA) {
                if (i > 0 && (i & 31) == 0) look(i), check();
                int page = __shfl_sync(0xffffffffu, ids, i & 31);
                const int slot = __shfl_sync(0xffffffffu, slots, i & 31);
                if (DOCS && page < 0) {
                    uint32_t some[1];
                    seen_keys(a, t, kb0 + i * Sp::kUnit, some);
                    if (lane == 0 && (some[0] & 0xFFFFu)) atomicOr(a.error, 4u);
                    page = 0;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, 2 * Sp::kSide + (a.stall && f == 0 ? 16 : 0));
#pragma unroll
                    for (int h = 0; h < ND; ++h) {
                        load_box(dst + h * kHalf, &maps.k, 64 * h, slot, head, page, bar);
                        load_box(dst + Sp::kSide + h * kHalf, &maps.v, 64 * h, slot, head, page, bar);
                    }
                }
            } else {
                // lane r < 16 finds row r
                const int key = kb0 + i * Sp::kUnit + (lane & 15);
                bool seen = key >= t.from && key < t.hi;
                if (holes) {
                    uint32_t some[1];
                    seen_keys(a, t, kb0 + i * Sp::kUnit, some);
                    seen = some[0] >> (lane & 15) & 1;
                }
                int page = 0, slot = 0;
                if (seen) {
                    int e;
                    page_of(a, key, e, slot);
                    page = pages[e];
                    if (page < 0 || page >= a.pages) {
                        atomicOr(a.error, 4u);
                        page = 0;
                    }
                }
                const uint32_t some = __ballot_sync(0xffffffffu, seen);
                constexpr int CPR = DP / 8;      // chunks of a row
#pragma unroll
                for (int j = 0; j < kBlock * CPR / 32; ++j) {
                    const int c = (lane + 32 * j) % CPR, r = (lane + 32 * j) / CPR;
                    const int64_t p = __shfl_sync(0xffffffffu, page, r), sl = __shfl_sync(0xffffffffu, slot, r);
                    const bool live = (some >> r & 1) && 8 * c < a.dim;
                    const uint32_t o = (c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                    // (a dead copy reads nothing; its address stays inside the cache)
                    const int64_t d = live ? 8 * c : 0;
                    copy16(dst + o, static_cast<const uint16_t *>(a.k) + p * a.k_page + sl * a.k_slot + head * a.k_head + d, live);
                    copy16(dst + Sp::kSide + o,
                           static_cast<const uint16_t *>(a.v) + p * a.v_page + sl * a.v_slot + head * a.v_head + d, live);
                }
                copies_arrive(bar);
            }
        };
        // row r of the tile: its token and its query head (divisions of small numbers)
        const int i0 = t.first ? t.first / a.group : 0, rem = t.first - i0 * a.group;
        const uint32_t inv = a.group < 32 ? 65536u / a.group + 1u : 0u;   // exact below 64
        auto token_of = [&](int r, int &hq) {
            const int x = rem + r, q = a.group < 32 ? static_cast<int>(x * inv >> 16) : (x >= a.group ? 1 : 0);
            hq = head * a.group + x - q * a.group;
            return i0 + q;
        };

        // ---- loads on their way: pages, queries (a warp per row), then the first slots
        if constexpr (TMA) look(0);
        constexpr int PER = R / WARPS;   // rows of a warp: w, w + WARPS, ..
        static_assert(PER * WARPS == R, "whole rows per warp");
        float x[PER][DP / 32];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int r = w + k * WARPS;
            int hq;
            const int tok = token_of(r, hq);
            const int64_t base = (t.tok0 + tok) * a.q_token + hq * a.q_head;
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                const int d = 32 * c + lane;
                x[k][c] = 0.0f;
                if (r < t.rows && d < a.dim) {
                    if (a.q_type == Q4K_F32) x[k][c] = static_cast<const float *>(a.q)[base + d];
                    else if (a.q_type == Q4K_F16) x[k][c] = __half2float(static_cast<const __half *>(a.q)[base + d]);
                    else x[k][c] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[base + d]);
                }
            }
        }
        if constexpr (TMA) check();
        const uint32_t first_fill = fills;
        fills += count;
        if (rg == 0) {
            if constexpr (TMA) fence_proxy_async_smem();   // (the ring may have held the previous tile's O)
            for (int i = 0; i < min(SLOTS, count); ++i) fill(i, first_fill + i);
        }

        // ---- the tile's rows: scale, visible range, fragments of Q
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int r = w + k * WARPS;
            const bool live = r < t.rows;
            int hq;
            const int tok = token_of(r, hq);
            float mx = 0.0f;
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) mx = fmaxf(mx, fabsf(x[k][c]));
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
                // d = 32 c + 16 i + 8 j + 2 t + b: half b of word 2 i + j of lane 4 (r % 8) + t
                float v = x[k][c] * up;
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    const uint32_t h = pack2(v, 0.0f, CT);
                    reinterpret_cast<uint16_t *>(&sh.q[p][r >> 3][c][4 * (r & 7) + ((lane >> 1) & 3)])
                        [2 * (lane >> 3) + (lane & 1)] = static_cast<uint16_t>(h & 0xFFFFu);
                    v -= unpack2(h, CT).x;
                }
            }
            if (lane == 0) {
                Range v{0, 0};
                if (live) v = token_range(a, t.seq, t.pos0 + tok, t.tok0 + tok, t.len);
                sh.lo[r] = v.lo, sh.hi[r] = v.hi;
                sh.pos[r] = tok;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                sh.scale[r] = (a.softcap > 0.0f ? a.scale / a.softcap : a.scale * kLog2e) * down;
                sh.slope[r] = live && a.slopes ? a.slopes[hq] * kLog2e : 0.0f;
            }
        }
        __syncthreads();

        int in_lo = 0, in_hi = 0x7FFFFFFF;   // keys that every live row sees
        for (int r = 0; r < t.rows; ++r) in_lo = max(in_lo, sh.lo[r]), in_hi = min(in_hi, sh.hi[r]);

        float m[NT][2], l[NT][2], o[NT][KS][4];   // o[..][i]: d = 16 i + g (+8), queries 2 t4 (+1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) m[nt][j] = -INFINITY, l[nt][j] = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
        }

        // a wait has timed out: the copies in flight land before the ring is used again
        auto wind_down = [&](int i) {
            if (lane == 0) atomicOr(a.error, 8u);
            for (int k = i; k < min(i + SLOTS, count); ++k)
                (void)mbar_wait_bounded(smem_u32(&sh.full[kg][(first_fill + k) % SLOTS]), ((first_fill + k) / SLOTS) & 1,
                                        kLandNs);
        };
        for (int i = 0; i < count; ++i) {
            const int kb = kb0 + i * Sp::kUnit;
            const uint32_t f = first_fill + i;
            const int slot = static_cast<int>(f % SLOTS);
            const uint32_t kt = ring + slot * 2 * Sp::kSide, vt = kt + Sp::kSide;
            const bool here = mbar_wait_bounded(smem_u32(&sh.full[kg][slot]), (f / SLOTS) & 1, a.wait_ns);
            good = __all_sync(0xffffffffu, here);
            if (!good) {
                wind_down(i);
                break;
            }
            auto zero_row = [&](int r) {
                if (lane < 8 * ND)
                    *reinterpret_cast<uint4 *>(sh.ring[kg] + slot * 2 * Sp::kSide + Sp::kSide + (lane >> 3) * kHalf + r * 128 +
                                               (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            };
            if (TMA && (kb < t.from || kb + kBlock > t.hi || holes)) {
                // rows of V that nothing sees: zero (by every warp that reads them)
                for (int r = 0; r < kBlock; ++r)
                    if (kb + r < t.from || kb + r >= t.hi) zero_row(r);
                if (holes) {
                    uint32_t some[1];
                    seen_keys(a, t, kb, some);
                    for (int r = 0; r < kBlock; ++r)
                        if (!(some[0] >> r & 1)) zero_row(r);
                }
                fence_proxy_async_smem();   // before a later copy into the slot
                __syncwarp();
            }

            if (8 * rg * NT < t.rows) {   // (this half may hold no rows)
                // ---- S^T
                // chains of their own: even and odd k-steps (one part), or the parts
                constexpr int CHAINS = PARTS > 1 ? PARTS : 2;
                float acc[NT][CHAINS][4] = {};
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    const int c = 2 * j + kch;
                    uint32_t kf[4];
                    ldmatrix4(kt + (c >> 3) * kHalf + krow * 128 + (((c & 7) ^ (krow & 7)) << 4), kf);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p) {
                            const uint2 b = reinterpret_cast<const uint2 *>(&sh.q[p][rg * NT + nt][j >> 1][lane])[j & 1];
                            mma_t<CT>(acc[nt][PARTS > 1 ? p : j & 1], kf[0], kf[1], kf[2], kf[3], b.x, b.y);
                        }
                }

                // (each step over all n8 tiles before the next: their chains run side by side)
                float s[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int r0 = 8 * (rg * NT + nt) + 2 * t4;
                    const float2 scl = *reinterpret_cast<const float2 *>(&sh.scale[r0]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x;
                        if constexpr (PARTS > 1) {
                            // an infinite key: the first part has its sign, the others may be 0 or of the other sign
                            float rest = acc[nt][PARTS - 1][j];
#pragma unroll
                            for (int p = PARTS - 2; p > 0; --p) rest += acc[nt][p][j];
                            x = fabsf(acc[nt][0][j]) < INFINITY ? acc[nt][0][j] + rest : acc[nt][0][j];
                        } else {
                            x = acc[nt][0][j] + acc[nt][1][j];
                        }
                        s[nt][j] = x * (j & 1 ? scl.y : scl.x);
                    }
                }
                if (a.softcap > 0.0f) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x = s[nt][j];
                            const float th = PARTS > 1 ? tanh_close(x) : 1.0f - 2.0f * rcp(ex2(2.0f * kLog2e * x) + 1.0f);
                            s[nt][j] = a.softcap * kLog2e * th;
                        }
                }
                if (a.slopes) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 8 * (rg * NT + nt) + 2 * t4 + (j & 1), key = kb + g + 8 * (j >> 1);
                            s[nt][j] -= sh.slope[r] * fabsf(static_cast<float>(t.pos0 + sh.pos[r] - key));
                        }
                }
                if (kb < in_lo || kb + kBlock > in_hi) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 8 * (rg * NT + nt) + 2 * t4 + (j & 1), key = kb + g + 8 * (j >> 1);
                            if (key < sh.lo[r] || key >= sh.hi[r]) s[nt][j] = -INFINITY;
                        }
                }
                float mx[NT][2], fa[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) mx[nt][j] = fmaxf(s[nt][j], s[nt][j + 2]);
#pragma unroll
                for (int hop = 4; hop < 32; hop <<= 1)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) mx[nt][j] = fmaxf(mx[nt][j], __shfl_xor_sync(0xffffffffu, mx[nt][j], hop));
                bool grown = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        mx[nt][j] = fmaxf(m[nt][j], mx[nt][j]);
                        grown |= mx[nt][j] != m[nt][j];
                        fa[nt][j] = mx[nt][j] == -INFINITY ? 1.0f : ex2(m[nt][j] - mx[nt][j]);
                        m[nt][j] = mx[nt][j];
                    }
                if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        l[nt][0] *= fa[nt][0], l[nt][1] *= fa[nt][1];
#pragma unroll
                        for (int q = 0; q < KS; ++q) {
                            o[nt][q][0] *= fa[nt][0], o[nt][q][1] *= fa[nt][1];
                            o[nt][q][2] *= fa[nt][0], o[nt][q][3] *= fa[nt][1];
                        }
                    }
                }
                uint32_t pb[NT][PARTS][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float base = mx[nt][j & 1] == -INFINITY ? 0.0f : mx[nt][j & 1] - kShift;
                        e[j] = ex2(s[nt][j] - base);
                        l[nt][j & 1] += e[j];
                    }
                    uint32_t p0[PARTS], p1[PARTS];
                    split2<CT, PARTS>(e[0], e[1], p0);
                    split2<CT, PARTS>(e[2], e[3], p1);
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) pb[nt][p][0] = transpose8(p0[p]), pb[nt][p][1] = transpose8(p1[p]);
                }

                // ---- O^T
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    const int c = 2 * j + vch;
                    uint32_t vf[4];
                    ldmatrix4_t(vt + (c >> 3) * kHalf + vrow * 128 + (((c & 7) ^ (vrow & 7)) << 4), vf);
                    if constexpr (PARTS > 1) {
                        // a block's sum by itself, added to O by an fp32 add: the MMA's own
                        // additions truncate, which over thousands of blocks is a bias
                        float sum[NT][4] = {};
#pragma unroll
                        for (int p = PARTS - 1; p >= 0; --p)   // small parts first
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_t<CT>(sum[nt], vf[0], vf[1], vf[2], vf[3], pb[nt][p][0], pb[nt][p][1]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int z = 0; z < 4; ++z) o[nt][j][z] += sum[nt][z];
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_t<CT>(o[nt][j], vf[0], vf[1], vf[2], vf[3], pb[nt][0][0], pb[nt][0][1]);
                    }
                }
            }
            __syncwarp();   // the slot has been read by every lane
            if (i + SLOTS < count) {
                if constexpr (RG > 1) {
                    if (lane == 0) mbar_arrive(smem_u32(&sh.empty[kg][slot]));
                    if (rg == 0) {   // .. of the group's other warp too
                        const bool free = mbar_wait_bounded(smem_u32(&sh.empty[kg][slot]), reads >> slot & 1, a.wait_ns);
                        reads ^= 1u << slot;
                        good = __all_sync(0xffffffffu, free);
                        if (!good) {
                            wind_down(i);
                            break;
                        }
                    }
                }
                if (rg == 0) fill(i + SLOTS, f + SLOTS);
            }
        }

        // ---- join the groups: each leaves O in its own ring
        if constexpr (RG > 1) __syncthreads();   // (its other warp may still be reading)
        float *red = reinterpret_cast<float *>(sh.ring[kg]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
                const int q = 8 * (rg * NT + nt) + 2 * t4 + j;
                if (g == 0) sh.m[kg][q] = m[nt][j], sh.l[kg][q] = l[nt][j];
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    red[q * Sh::kRed + 16 * i + g] = o[nt][i][j];
                    red[q * Sh::kRed + 16 * i + 8 + g] = o[nt][i][j + 2];
                }
            }
        __syncthreads();
        const bool split = a.cluster ? a.cluster > 1 : todo < t.units;
        const bool send = a.cluster > 1;
        constexpr int DQ = DP / 4;                           // column quads
        const int share = send ? (DQ + a.cluster - 1) / a.cluster : DQ;   // of a rank
        if (send) {
            cluster_wait_acquire();   // every CTA of the cluster has started
            // the row statistics of this CTA, to every rank
            const int rank = cta % a.cluster;
            for (int i = tid; i < R * a.cluster; i += THREADS) {
                const int r = i % R;
                float mx = -INFINITY, ls = 0.0f;
#pragma unroll
                for (int k = 0; k < KG; ++k) mx = fmaxf(mx, sh.m[k][r]);
#pragma unroll
                for (int k = 0; k < KG; ++k) ls += sh.l[k][r] * weight(sh.m[k][r], mx);
                st_shared_cluster_v2(map_shared_rank(smem_u32(&sh.stat[rank][r]), i / R), mx, ls);
            }
        }
        float *part = a.part + part_slot(cta, off == 0) * (R * (DP + 2));
        for (int i = tid; i < t.rows * (DP / 4); i += THREADS) {
            const int r = i / (DP / 4), d = 4 * (i % (DP / 4));
            float mx = -INFINITY, ls = 0.0f;
#pragma unroll
            for (int k = 0; k < KG; ++k) mx = fmaxf(mx, sh.m[k][r]);
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < KG; ++k) {
                const float f = weight(sh.m[k][r], mx);
                const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sh.ring[k]) + r * Sh::kRed + d);
                ls += f * sh.l[k][r];
                v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
            }
            if (d >= a.dim) continue;
            if (send) {   // to the rank that owns the columns
                const int q = d / 4, to = q / share;
                st_shared_cluster_v4(map_shared_rank(smem_u32(&sh.sent[(cta % a.cluster * R + r) * share + q - to * share]), to), v);
            } else if (split) {
                reinterpret_cast<float4 *>(part)[d / 4 * R + r] = v;
                if (d == 0) part[R * DP + r] = mx, part[R * DP + R + r] = ls;
            } else {
                int hq;
                const int tok = token_of(r, hq);
                finish_row(a, t.tok0 + tok, hq, d, v, mx, ls, kShift);
            }
        }

        if (send) {
            // ---- a cluster: each CTA adds its columns over the ranks, in key order
            __syncthreads();
            cluster_sync_all();
            const int rank = cta % a.cluster;
            for (int i = tid; i < t.rows * share; i += THREADS) {
                const int r = i / share, d = 4 * (rank * share + i - r * share);
                if (d >= a.dim) continue;   // (the last rank's share may end past the head)
                float mx = -INFINITY, ls = 0.0f;
                for (int c = 0; c < a.cluster; ++c) mx = fmaxf(mx, sh.stat[c][r].x);
                float4 v = make_float4(0, 0, 0, 0);
                for (int c = 0; c < a.cluster; ++c) {
                    const float f = weight(sh.stat[c][r].x, mx);
                    const float4 x = sh.sent[c * R * share + i];
                    ls += f * sh.stat[c][r].y;
                    v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
                }
                int hq;
                const int tok = token_of(r, hq);
                finish_row(a, t.tok0 + tok, hq, d, v, mx, ls, kShift);
            }
        } else if (split && off == 0 && tid == 0) {
            a.joint[cta] = Joint{t.tok0, t.first, t.rows, head, cta, share_owner(total, n, u0 + t.units - 1)};
        }
        if (a.cluster) break;   // one tile per cluster (a rank's share of it may be empty)
        u += todo;
        __syncthreads();   // the tile's shared data is done with
    }
}

// What q4k_attn_plan.h chose for a call.
struct Choice {
    bool chunk;    // the many-rows kernel
    int rows;      // few-rows: query rows of a tile
    int cluster;   // few-rows: CTAs of a cluster per tile, 0: split over the SMs
};

struct RowsLaunch {
    Args args;
    Choice choice;
    int device, sms, parts_many;   // parts_many: fp32 queries or outputs, or a 16-bit type that is not the cache's
    bool boxes;            // pages and strides that TMA boxes of 16 slots can take
    cudaStream_t stream;
};
cudaError_t clusters_at_once(int (&n)[kMaxCluster + 1]);
// The kernel of one cache type, without and with holes (each in a translation unit of its own).
cudaError_t launch_rows_f16(const RowsLaunch &l);
cudaError_t launch_rows_bf16(const RowsLaunch &l);
cudaError_t launch_rows_docs_f16(const RowsLaunch &l);
cudaError_t launch_rows_docs_bf16(const RowsLaunch &l);

}  // namespace attn
}  // namespace q4k
