// q4k_attn_chunk.cuh -- attention of many query rows per cache head (prompt
// chunks) on the tcgen05 tensor cores, keys and values by TMA from their pages.
//
// 4 dim flops per (row, key) against 4 dim bytes per key and 256-row tile: the
// tensor cores bound it (two 128 x 128 x 128 products a step and half tile, 512
// cycles each), with one exponential per (row, key) beside them.
//
// CTA: tiles of whole tokens, up to 256 query rows, as two halves of 128 (the
// MMA's M); one CTA per SM, persistent over its share of the call's units (128
// keys each).
//   * warps 0-3 and 4-7: softmax of a half, a thread per row: S from tensor
//     memory (128 values), mask, maximum, exponentials, P as 16-bit pairs back
//     into the columns of S; at the end of a tile O out of tensor memory.
//   * warp 8 issues the MMAs: S = Q K^T (both from shared memory, K-major) and
//     O += P V (P from tensor memory, V from shared memory as it lies, rows of
//     keys: MN-major).  The halves alternate, so one half's softmax runs
//     under the other's products, and P is taken up in two parts.
//   * warp 9 walks the tiles and tells the others (a ring of two descriptors),
//     loads the tile's queries (a TMA box of its tokens and the group's heads) as
//     soon as the last scores of the tile before are done, and the keys, two
//     stages of 128; warp 10 loads the values, two stages: a lane per page piece
//     looks the page up and issues its boxes.
// Softmax threads take 200 registers (a row of S and change), the others 96.
// Tensor memory, all 512 columns: S (and P) of the halves, O of the halves.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the
// one in use (exponents relative to an older maximum stay exact in fp32 and
// within the range of 16 bits), which after the first tiles is rare.  When S of
// step i is complete, so is the O of step i - 1 (MMAs complete in order), so
// the rescaling waits for nothing.
//
// Slots that nothing of the tile sees may hold NaN: scores are replaced, not
// added to, and the rows of V outside the tile's keys, or in a hole that a document
// mask leaves between them, are zeroed in shared memory before they meet P = 0.
// A widened 8-bit cache (MODE bit 3; q4k_attn_widen.cu): keys and values are codes, or
// codes over a power of two, in fp16, in pages of 128 that follow each other; each piece of
// 16 of them has a factor.  Warp 11 hands the factors of the units on, some ahead.  The
// keys' multiply the scores, the values' join the exponents of P by their log2, over the
// largest so far, by which O is rescaled as by a maximum; the sum of a piece loses it
// again.  That is a multiplication a piece and row, and no instruction a score more; three
// chunks of 512 over 4096 take 79 us where the 16-bit kernel takes 69, 2048 tokens over
// 14336 347 where it takes 300 (each launch by itself).  Pieces that no row of the tile sees
// have no factor, whatever lies there.
//
// Every wait is bounded in time: on a timeout the CTA sets bit 3 of the error word,
// stops, waits (bounded) for its copies and products in flight, frees its tensor
// memory and returns.
//
// Measured (device): 2048 tokens of 32 / 8 bf16 heads over 14336 + 2048 positions 310
// to 330 us, 1560 to 1660 TFLOP/s = 80 to 85 % of the measured matmul, tensor pipe
// 76 % active (784 us with capped scores) (S read twice in pieces 451; eight query loads at a time 410; one
// pipeline over tiles, a row of S in registers, P in two parts 340); three chunks of
// 512 over 4096 81 us, of which 21 are start and join.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "q4k_attn.cuh"
#include "q4k_codes.cuh"
#include "ptx.cuh"

namespace q4k {
namespace attn {

constexpr int kChunkRows = 256;              // query rows of a tile at most
constexpr int kChunkKeys = 128;              // keys of a unit
constexpr int kChunkThreads = 384;           // two softmax warpgroups; MMA, key, value and idle warp
constexpr int kMmaWarp = 8, kKeyWarp = 9, kValueWarp = 10, kFactorWarp = 11;
constexpr int kStages = 4;
// 256 x 200 + 128 x 96 registers, within the 384 x 168 of the launch; a widened cache's
// factors take more beside a row of S: 256 x 208 + 128 x 88
constexpr int softmax_regs(int mode) { return mode & 8 ? 208 : 200; }
constexpr int other_regs(int mode) { return mode & 8 ? 88 : 96; }

// A CTA's part of one tile, as the key warp found it.
struct Work {
    Tile t;
    int head, off, todo, last;   // units [off, off + todo) of the tile; the CTA that holds the tile's last unit
};

// The factors of a unit's pieces of 16: of the keys; of the values over 2^top as log2, and
// one over that; by how much top has grown since the tile's (or this part's) unit before.
struct UnitFactors {
    float key[8], value[8], undo[8];
    int top, grown;
};
constexpr int kUnitsAhead = 4;

template <int DP>
struct ChunkShared {
    static constexpr int kHalf = 128 * 128;                    // bytes: 128 rows of 64 elements
    static constexpr int kTile = kHalf * (DP / 64);            // 128 rows of DP elements
    uint8_t q[2 * kTile];                                      // [dim / 64][256 rows][64]
    uint8_t kv[kStages * kTile];
    uint8_t out[8][32 * 64];                                   // a warp's rows on their way out, 32 columns at a time
    SplitShared<kChunkThreads> plan;
    unsigned long long full[kStages], empty[kStages], s_full[2], p_ready[2][2], o_done[2], q_full, q_empty, edge, drained;
    unsigned long long work_full[2], work_empty[2];
    Work work[2];
    alignas(16) uint32_t seen[2][kChunkKeys / 32];   // (tiles with holes) of the key and the value warp
    unsigned long long factors_full[kUnitsAhead], factors_empty[kUnitsAhead];
    UnitFactors factors[kUnitsAhead];
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void tm_ld32(uint32_t addr, float *r)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr));
}

__device__ __forceinline__ void tm_ld16(uint32_t addr, float *r)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr));
}

__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t *u)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(u[0]),
        "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
        "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(addr)
        : "memory");
}

// Waits for the loads issued so far; the registers of the one that is about to be
// used are operands, so that nothing that reads them moves ahead of the wait.
__device__ __forceinline__ void tm_wait_ld32(float *r)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]),
                   "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]),
                   "+r"(u[15]), "+r"(u[16]), "+r"(u[17]), "+r"(u[18]), "+r"(u[19]), "+r"(u[20]), "+r"(u[21]),
                   "+r"(u[22]), "+r"(u[23]), "+r"(u[24]), "+r"(u[25]), "+r"(u[26]), "+r"(u[27]), "+r"(u[28]),
                   "+r"(u[29]), "+r"(u[30]), "+r"(u[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tm_wait_ld16(float *r)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]),
                   "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tm_here32(float *r)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(""
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]),
                   "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]),
                   "+r"(u[15]), "+r"(u[16]), "+r"(u[17]), "+r"(u[18]), "+r"(u[19]), "+r"(u[20]), "+r"(u[21]),
                   "+r"(u[22]), "+r"(u[23]), "+r"(u[24]), "+r"(u[25]), "+r"(u[26]), "+r"(u[27]), "+r"(u[28]),
                   "+r"(u[29]), "+r"(u[30]), "+r"(u[31])
                 :
                 : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// The largest of three (NaN only if all are).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Query rows: 64 elements of the group's heads of some tokens.
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, int d, int head, int token, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(d), "r"(head), "r"(token), "r"(bar)
        : "memory");
}

// Issued by one elected lane of a converged warp (the loop's arithmetic stays
// warp-uniform that way).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle, rows of 128 bytes in atoms
// of 8 rows (1024 bytes).  K-major: `lead` is not used.  MN-major (V): `lead` is
// the distance of the next 64 elements of a row, the atoms follow along K.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lead)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

// Instruction descriptor, kind::f16, fp32 accumulators, M = 128.
template <int CT>
constexpr uint32_t chunk_idesc(int n, bool b_mn_major)
{
    return (1u << 4) | (CT == Q4K_BF16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// fp16 weights are kept at 2^6 and below 2^14; bf16 has range to spare.
template <int CT>
constexpr float chunk_shift()
{
    return CT == Q4K_F16 ? 6.0f : 0.0f;
}

// MODE bit 0: capped scores, bit 1: distance bias, bit 2 (DOCS): a causal call with
// kv_start, whose tiles may have holes (its code in every instance cost 2048 tokens
// over 14336 positions 2 %), bit 3: a widened 8-bit cache.
template <int CT, int DP, int MODE>
__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_kernel(const __grid_constant__ CacheMaps maps, const __grid_constant__ CUtensorMap qmap, const Args a, const int box)
{
    using Sh = ChunkShared<DP>;
    constexpr int kHalf = Sh::kHalf, kTile = Sh::kTile, ND = DP / 64;
    constexpr bool DOCS = MODE & 4, WIDE = MODE & 8;
    constexpr float kShift = chunk_shift<CT>();
    constexpr float kLazy = 8.0f;
    extern __shared__ uint8_t smem_raw[];
    Sh &sh = *reinterpret_cast<Sh *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int tokens = kChunkRows / a.group;   // of a tile

    if (w == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&sh.full[i]), 1), mbar_init(smem_u32(&sh.empty[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.s_full[i]), 1);
            mbar_init(smem_u32(&sh.p_ready[i][0]), 128);
            mbar_init(smem_u32(&sh.p_ready[i][1]), 128);
            mbar_init(smem_u32(&sh.o_done[i]), 1);
            mbar_init(smem_u32(&sh.work_full[i]), 1);
            mbar_init(smem_u32(&sh.work_empty[i]), WIDE ? 11 : 10);   // the MMA, value (factor) and eight softmax warps
        }
        if constexpr (WIDE)
            for (int i = 0; i < kUnitsAhead; ++i) mbar_init(smem_u32(&sh.factors_full[i]), 1), mbar_init(smem_u32(&sh.factors_empty[i]), 8);
        mbar_init(smem_u32(&sh.q_full), 1);
        mbar_init(smem_u32(&sh.q_empty), 1);
        mbar_init(smem_u32(&sh.edge), 1);
        mbar_init(smem_u32(&sh.drained), 1);
        fence_barrier_init();
        sh.abort = 0;
    }
    if (tid == 32) prefetch_tensormap(&maps.k), prefetch_tensormap(&maps.v), prefetch_tensormap(&qmap);
    tm_fence_before();
    pdl_launch_dependents();
    pdl_wait();   // (everything below may come from the kernel before)
    Split<kChunkKeys, kChunkThreads, kChunkKeys, DOCS> plan(a, sh.plan, tokens * a.group);   // synchronises the CTA
    plan.scan();
    tm_fence_after();
    const uint32_t tm = sh.tmem;

    // Waits for a phase, whole warps together; false: the CTA winds down.
    volatile int *abort = &sh.abort;
    auto wait_lane = [&](uint32_t b, uint32_t parity) -> bool {
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t i = 1;; ++i) {
            if (mbar_try_wait_sleep(b, parity, 20000u)) return true;
            if ((i & 15u) == 0u) {
                if (*abort) return false;
                if (globaltimer_ns() - t0 > a.wait_ns) {
                    *abort = 1;
                    atomicOr(a.error, 8u);
                    return false;
                }
            }
        }
    };
    auto wait = [&](unsigned long long &bar, uint32_t parity) -> bool {
        const uint32_t b = smem_u32(&bar);
        const bool done = mbar_try_wait(b, parity) || wait_lane(b, parity);
        return __all_sync(0xffffffffu, done);
    };

    const int64_t total = static_cast<int64_t>(plan.per_head) * a.kv_heads;
    const int n = sharers(total, gridDim.x);
    const int cta = blockIdx.x;
    int64_t u = 0, u_end = 0;
    if (cta < n) u = share_begin(total, n, cta), u_end = share_begin(total, n, cta + 1);
    const bool known = plan.hand_out(per_head_rest(u, plan.per_head));   // the first tile
    if (tid == 0) a.joint[cta].rows = 0;

    // The k-th part of a tile of this CTA, out of the ring; all lanes of a warp.
    auto next_work = [&](int k, Work &item) -> bool {
        if (!wait(sh.work_full[k & 1], (k >> 1) & 1)) return false;
        item = sh.work[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.work_empty[k & 1]));
        return true;
    };

    if (w == kKeyWarp || w == kValueWarp) {
        // ------------------------------------------------------------ loads
        regs_dec<other_regs(MODE)>();
        const bool values = w == kValueWarp;
        const CUtensorMap *map = values ? &maps.v : &maps.k;
        int unit = 0, edges = 0, k = 0;   // this warp's stage of unit i: 2 (i % 2), + 1 for values
        bool ok = true, q_sent = false;
        const int per = kChunkKeys / box;
        auto queries = [&](const Work &item) {
            if (lane == 0) {
                mbar_arrive_expect_tx(smem_u32(&sh.q_full), tokens * a.group * 128 * ND);
#pragma unroll
                for (int h = 0; h < ND; ++h)
                    load_rows(smem_u32(sh.q + h * 2 * kHalf), &qmap, 64 * h, item.head * a.group,
                              item.t.tok0 + item.t.first / a.group, smem_u32(&sh.q_full));
            }
            q_sent = true;
            __syncwarp();
        };
        for (; ok; ++k) {
            Work item;
            if (values) {
                ok = next_work(k, item);
                if (!ok || item.todo == 0) break;
            } else {
                // the key warp finds the tiles and tells the others (todo = 0: no more)
                if (k > 1 && !(ok = wait(sh.work_empty[k & 1], ((k >> 1) - 1) & 1))) break;
                item.todo = 0;
                if (u < u_end) {
                    item.head = static_cast<int>(quotient(u, plan.per_head));
                    if (k == 0 && known) item.t = sh.plan.first, item.off = sh.plan.offset;
                    else item.t = plan.locate(static_cast<uint32_t>(u - static_cast<int64_t>(item.head) * plan.per_head), item.off);
                    item.todo = static_cast<int>(min(static_cast<int64_t>(item.t.units - item.off), u_end - u));
                    item.last = share_owner(total, n, u - item.off + item.t.units - 1);
                    u += item.todo;
                }
                if (lane == 0) {
                    sh.work[k & 1] = item;
                    mbar_arrive(smem_u32(&sh.work_full[k & 1]));
                }
                __syncwarp();
                if (item.todo == 0) break;
            }
            const bool holes = DOCS && (item.t.seq & kHoles);
            if (DOCS) item.t.seq &= ~kHoles;
            const Tile &t = item.t;
            const int32_t *pages = a.page_table + static_cast<int64_t>(t.seq) * a.table_stride;
            if (!values && k == 0) queries(item);
            for (int i = 0; i < item.todo && ok; ++i, ++unit) {
                const int kb = t.lo + (item.off + i) * kChunkKeys;
                const int stage = 2 * (unit & 1) + (values ? 1 : 0);
                // lane j: piece j of the tile
                const int key = kb + lane * box;
                bool live = lane < per && key + box > t.from && key < t.hi;
                if (holes) {   // the keys that some row sees: no others are looked up, and their values are zeroed below
                    uint32_t seen[kChunkKeys / 32];
                    seen_keys(a, t, kb, seen);
                    if (lane == 0) *reinterpret_cast<uint4 *>(sh.seen[values]) = make_uint4(seen[0], seen[1], seen[2], seen[3]);
                    __syncwarp();
                    live = false;
                    for (int z = 0; z < box && lane < per; z += 16)
                        live |= (sh.seen[values][(lane * box + z) >> 5] >> ((lane * box + z) & 31) & 0xFFFFu) != 0;
                    __syncwarp();
                }
                int page = 0, slot = 0;
                if (live) {
                    int e;
                    page_of(a, key, e, slot);
                    if constexpr (WIDE) {
                        page = t.seq * a.table_pages + e;
                    } else {
                        page = pages[e];
                        if (page < 0 || page >= a.pages) {
                            atomicOr(a.error, 4u);
                            live = false;
                        }
                    }
                }
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * static_cast<uint32_t>(box) * 128u * ND;
                if (unit > 1 && !(ok = wait(sh.empty[stage], ((unit >> 1) - 1) & 1))) break;
                uint8_t *dst = sh.kv + stage * kTile;
                const bool clean = values && (kb < t.from || kb + kChunkKeys > t.hi || holes);
                unsigned long long &bar = clean ? sh.edge : sh.full[stage];
                if (lane == 0) mbar_arrive_expect_tx(smem_u32(&bar), bytes + (a.stall && !values && unit == 0 ? 16 : 0));
                __syncwarp();
                if (live) {
#pragma unroll
                    for (int h = 0; h < ND; ++h)
                        load_box(smem_u32(dst + h * kHalf + lane * box * 128), map, 64 * h, slot, item.head, page,
                                 smem_u32(&bar));
                }
                if (i == 0 && k > 0 && !values) {
                    // the tile's queries, once the last scores of the tile before are done
                    if (!(ok = wait(sh.q_empty, (k - 1) & 1))) break;
                    queries(item);
                }
                if (clean) {
                    // zero the rows that nothing of the tile sees, then hand the stage on
                    if (!(ok = wait(sh.edge, edges & 1))) break;
                    ++edges;
                    const int r0 = max(0, t.from - kb), r1 = min(kChunkKeys, t.hi - kb);
                    auto zero_row = [&](int r) {
                        if (lane < 8 * ND)
                            *reinterpret_cast<uint4 *>(dst + (lane >> 3) * kHalf + r * 128 + (lane & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    };
                    for (int r = 0; r < kChunkKeys; ++r) {
                        if (r >= r0 && r < r1) continue;
                        zero_row(r);
                    }
                    if (holes)
#pragma unroll 1
                        for (int r = r0; r < r1; ++r)
                            if (!(sh.seen[1][r >> 5] >> (r & 31) & 1)) zero_row(r);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.full[stage]));
                }
            }
        }
        // every copy issued lands before the CTA exits (another warp may wind down without having
        // waited for it): this warp's last two stages, one that it has begun, the queries
        for (int i = max(0, unit - 2); i < unit + (ok ? 0 : 1); ++i)
            (void)mbar_wait_bounded(smem_u32(&sh.full[2 * (i & 1) + (values ? 1 : 0)]), (i >> 1) & 1, kLandNs);
        if (!ok && values) (void)mbar_wait_bounded(smem_u32(&sh.edge), edges & 1, kLandNs);
        if (q_sent) (void)mbar_wait_bounded(smem_u32(&sh.q_full), (k + 1) & 1, kLandNs);   // (of tile k - 1)
        if (q_sent && !ok) (void)mbar_wait_bounded(smem_u32(&sh.q_full), k & 1, kLandNs);
    } else if (w == kMmaWarp) {
        // ------------------------------------------------------------ products
        regs_dec<other_regs(MODE)>();
        constexpr uint32_t id_s = chunk_idesc<CT>(kChunkKeys, false), id_o = chunk_idesc<CT>(DP, true);
        const uint32_t q0 = smem_u32(sh.q), kv0 = smem_u32(sh.kv);
        int stage = 0;
        uint32_t round = 0, steps[2] = {0, 0};
        bool ok = true;
        auto take = [&](uint32_t &addr) -> bool {   // next stage of the ring
            if (!wait(sh.full[stage], round & 1)) return false;
            addr = kv0 + stage * kTile;
            return true;
        };
        auto next = [&]() {
            if (++stage == kStages) stage = 0, ++round;
        };
        auto scores = [&](int h, uint32_t k) {
#pragma unroll
            for (int j = 0; j < DP / 16; ++j)
                mma_ss(tm + 128 * h, tile_desc(q0 + (j >> 2) * 2 * kHalf + h * kHalf + (j & 3) * 32, 16),
                       tile_desc(k + (j >> 2) * kHalf + (j & 3) * 32, 16), id_s, j > 0);
            mma_commit(smem_u32(&sh.s_full[h]));
        };
        for (int k = 0; ok; ++k) {
            Work item;
            ok = next_work(k, item);
            if (!ok || item.todo == 0) break;
            const int todo = item.todo, halves = item.t.rows > 128 ? 2 : 1;
            uint32_t kt = 0, vt = 0;
            ok = wait(sh.q_full, k & 1) && take(kt);
            if (!ok) break;
            tm_fence_after();
            for (int h = 0; h < halves; ++h) scores(h, kt);
            mma_commit(smem_u32(&sh.empty[stage]));
            if (todo == 1) mma_commit(smem_u32(&sh.q_empty));
            next();
            for (int i = 0; i < todo && ok; ++i) {
                ok = take(vt);
                const int vstage = stage;
                next();
                const bool more = i + 1 < todo;
                for (int h = 0; h < halves && ok; ++h) {
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        ok = ok && wait(sh.p_ready[h][part], steps[h] & 1);
                        if (!ok) break;
                        tm_fence_after();
#pragma unroll
                        for (int j = 4 * part; j < 4 * part + 4; ++j)
                            mma_ts(tm + 256 + 128 * h, tm + 128 * h + 8 * j, tile_desc(vt + j * 2048, kHalf), id_o,
                                   i > 0 || j > 0);
                    }
                    if (!ok) break;
                    ++steps[h];
                    if (!more) mma_commit(smem_u32(&sh.o_done[h]));
                    if (h == halves - 1) mma_commit(smem_u32(&sh.empty[vstage]));
                    if (more) {
                        if (h == 0) ok = take(kt);
                        if (!ok) break;
                        tm_fence_after();
                        scores(h, kt);
                        if (h == halves - 1) {
                            mma_commit(smem_u32(&sh.empty[stage]));
                            if (i + 2 == todo) mma_commit(smem_u32(&sh.q_empty));
                            next();
                        }
                    }
                }
            }
        }
    } else if (w < 8) {
        // ------------------------------------------------------------ softmax
        regs_inc<softmax_regs(MODE)>();
        const int h = w >> 2, row = tid;                // row of the tile: half h, TMEM lane tid % 128
        const uint32_t lane_base = static_cast<uint32_t>(w & 3) << 21;   // 32 (w % 4) lanes, in bits 16..
        const uint32_t ts = tm + lane_base + 128 * h, to = tm + lane_base + 256 + 128 * h;
        uint32_t steps = 0, done = 0;
        int unit = 0;                                   // (WIDE) units of this CTA so far
        bool ok = true;
        // masked scores are -inf: keep their product with the scale -inf when the scale is 0
        const float c = (MODE & 1) ? a.scale / a.softcap : fmaxf(a.scale * kLog2e, 1e-30f);
        for (int k = 0; ok; ++k) {
            Work item;
            ok = next_work(k, item);
            if (!ok || item.todo == 0) break;
            if (DOCS) item.t.seq &= ~kHoles;
            const Tile &t = item.t;
            const int head = item.head, off = item.off, todo = item.todo;
            if (t.rows <= 128 * h) {
                if constexpr (WIDE) {   // (the units are not this warp's, but it counts for their places)
                    for (int i = 0; i < todo && ok; ++i, ++unit) {
                        ok = wait(sh.factors_full[unit % kUnitsAhead], (unit / kUnitsAhead) & 1);
                        if (ok && lane == 0) mbar_arrive(smem_u32(&sh.factors_empty[unit % kUnitsAhead]));
                    }
                }
                continue;
            }

            // ---- this row's keys
            const uint32_t gr = t.first + row, tok = gr / static_cast<uint32_t>(a.group);
            const int hq = head * a.group + static_cast<int>(gr - tok * a.group);
            const bool live = row < t.rows;
            int lo = 0, hi = 0;
            if (live) {
                const Range r = token_range(a, t.seq, t.pos0 + tok, t.tok0 + tok, t.len);
                lo = r.lo, hi = r.hi;
            }
            // keys that every live row of the warp sees need no mask
            int in_lo = live ? lo : 0, in_hi = live ? hi : 0x7FFFFFFF;
            in_lo = __reduce_max_sync(0xffffffffu, in_lo);
            in_hi = __reduce_min_sync(0xffffffffu, in_hi);
            const float slope = (MODE & 2) && live ? a.slopes[hq] * kLog2e : 0.0f;
            const int rel = live ? t.pos0 + static_cast<int>(tok) : 0;   // position, for the distance

            float m = -INFINITY, l = 0.0f;   // maximum in use (of c s, log2) and sum
            float cq = c;                    // (WIDE) with the power of two of the row's queries
            int top = 0;                     // (WIDE) O is over 2^top
            if (WIDE && live && a.row_scale) cq = c * a.row_scale[static_cast<int64_t>(t.tok0 + tok) * a.heads + hq];
            for (int i = 0; i < todo; ++i) {
                const int kb = t.lo + (off + i) * kChunkKeys;
                ok = wait(sh.s_full[h], steps & 1);
                if (!ok) break;
                ++steps;
                tm_fence_after();
                float s[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tm_ld32(ts + 32 * q, s[q]);
                tm_wait_ld32(s[0]);
#pragma unroll
                for (int q = 1; q < 4; ++q) tm_here32(s[q]);
                float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                int grown = 0;               // (WIDE) by which the unit raises top
                const UnitFactors *fac = &sh.factors[unit % kUnitsAhead];
                if constexpr (WIDE) {
                    ok = wait(sh.factors_full[unit % kUnitsAhead], (unit / kUnitsAhead) & 1);
                    if (!ok) break;
                    grown = fac->grown, top = fac->top;
                }
                // the factor of the scores of columns 32 q + 16 b and on
                // (WIDE: never 0, a score that is masked out has to stay -inf)
                auto score = [&](int q, int b) { return WIDE ? fmaxf(cq * fac->key[2 * q + b], 1e-38f) : c; };
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float *v = s[q];
                    const float c0 = score(q, 0), c1 = WIDE ? score(q, 1) : c0;
                    if (MODE & 1) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = a.softcap * kLog2e * (1.0f - 2.0f * rcp(ex2(2.0f * kLog2e * (v[j] * (j < 16 ? c0 : c1))) + 1.0f));
                    }
                    if (MODE & 2) {
                        const float d0 = static_cast<float>(rel - kb - 32 * q);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = fmaf(-slope, fabsf(d0 - static_cast<float>(j)), (MODE & 1) ? v[j] : v[j] * (j < 16 ? c0 : c1));
                    }
                    if (kb < in_lo || kb + kChunkKeys > in_hi) {
                        const int a0 = lo - kb - 32 * q, a1 = hi - kb - 32 * q;
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = j >= a0 && j < a1 ? v[j] : -INFINITY;
                    }
                    if constexpr (WIDE && !(MODE & 3)) {   // a maximum for each factor
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const float *u = v + 16 * b;
                            const float p0 = max3(u[0], u[1], u[2]), p1 = max3(u[3], u[4], u[5]), p2 = max3(u[6], u[7], u[8]),
                                        p3 = max3(u[9], u[10], u[11]), p4 = max3(u[12], u[13], u[14]);
                            x[q] = fmaxf(x[q], fmaxf(max3(p0, p1, p2), max3(p3, p4, u[15])) * (b ? c1 : c0));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
#pragma unroll
                            for (int z = 0; z < 4; ++z) x[z] = max3(x[z], v[j + 2 * z], v[j + 2 * z + 1]);
                        }
                    }
                }
                const float mul = (MODE & 3) ? 1.0f : c;
                const float mx = fmaxf(max3(x[0], x[1], x[2]), x[3]) * (WIDE ? 1.0f : mul);
                float f = 1.0f;
                if (mx > m + kLazy || m == -INFINITY) {
                    // (m = mx = -inf: everything masked so far, l and O are zero)
                    f = mx == m ? 1.0f : ex2(m - mx);
                    m = mx;
                }
                if (i > 0 && (__any_sync(0xffffffffu, f != 1.0f) || (WIDE && grown))) {
                    l *= f;
                    if constexpr (WIDE) f *= two_to(max(-grown, -126));
#pragma unroll
                    for (int j = 0; j < DP / 16; ++j) {
                        float o[16];
                        tm_ld16(to + 16 * j, o);
                        tm_wait_ld16(o);
#pragma unroll
                        for (int z = 0; z < 16; ++z) o[z] *= f;
                        tm_st16(to + 16 * j, reinterpret_cast<const uint32_t *>(o));
                    }
                }
                const float base = m == -INFINITY ? 0.0f : m - kShift;
                const uint64_t mul2 = pair(mul, mul), base2 = pair(-base, -base);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t p[16];
                    // (WIDE: P times the values' factor of its piece over 2^top; the sum loses it again)
                    uint64_t mul_a = mul2, mul_b = mul2, base_a = base2, base_b = base2;
                    if constexpr (WIDE) {
                        const float x0 = fac->value[2 * q] - base, x1 = fac->value[2 * q + 1] - base;
                        base_a = pair(x0, x0), base_b = pair(x1, x1);
                        sum[0] = sum[1] = 0;
                        if (!(MODE & 3)) {
                            const float m0 = score(q, 0), m1 = score(q, 1);
                            mul_a = pair(m0, m0), mul_b = pair(m1, m1);
                        }
                    }
#pragma unroll
                    for (int z = 0; z < 16; ++z) {
                        float e0, e1;
                        unpair(fma2(pair(s[q][2 * z], s[q][2 * z + 1]), z < 8 ? mul_a : mul_b, z < 8 ? base_a : base_b), e0, e1);
                        e0 = ex2(e0), e1 = ex2(e1);
                        uint64_t &add = sum[WIDE ? z >> 3 : z & 1];
                        add = add2(add, pair(e0, e1));
                        p[z] = pack2(e0, e1, CT);
                    }
                    if constexpr (WIDE) {
                        float l0, l1;
                        unpair(sum[0], l0, l1);
                        l = fmaf(l0 + l1, fac->undo[2 * q], l);
                        unpair(sum[1], l0, l1);
                        l = fmaf(l0 + l1, fac->undo[2 * q + 1], l);
                    }
                    tm_st16(ts + 16 * q, p);
                    if (q & 1) {   // 64 keys of P: the products can start on them
                        tm_wait_st();
                        tm_fence_before();
                        mbar_arrive(smem_u32(&sh.p_ready[h][q >> 1]));
                    }
                }
                if constexpr (WIDE) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.factors_empty[unit % kUnitsAhead]));
                    ++unit;
                } else {
                    float l0, l1;
                    unpair(add2(sum[0], sum[1]), l0, l1);
                    l += l0 + l1;
                }
            }
            if (!ok) break;
            const float back = WIDE ? two_to(top) : 1.0f;   // O's power of two

            // ---- O: divide and store, or leave a partial result ([dim / 4][row] quads, maxima, sums)
            ok = wait(sh.o_done[h], done & 1);
            if (!ok) break;
            ++done;
            tm_fence_after();
            if (todo < t.units) {
                float *part = a.part + part_slot(cta, off == 0) * (kChunkRows * (DP + 2));
#pragma unroll
                for (int j = 0; j < DP / 32; ++j) {
                    float o[32];
                    tm_ld32(to + 32 * j, o);
                    tm_wait_ld32(o);
                    if constexpr (WIDE)
#pragma unroll
                        for (int z = 0; z < 32; ++z) o[z] *= back;
                    if (live) {
#pragma unroll
                        for (int z = 0; z < 8; ++z)
                            reinterpret_cast<float4 *>(part)[(8 * j + z) * kChunkRows + row] =
                                make_float4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]);
                    }
                }
                if (live) part[kChunkRows * DP + row] = m, part[kChunkRows * (DP + 1) + row] = l;
                if (off == 0 && tid == 0) a.joint[cta] = Joint{t.tok0, t.first, t.rows, head, cta, item.last};
            } else {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                // through shared memory, so that four lanes write 64 bytes of a row together
                uint8_t *box_out = sh.out[w];
#pragma unroll
                for (int j = 0; j < DP / 32; ++j) {
                    float o[32];
                    tm_ld32(to + 32 * j, o);
                    tm_wait_ld32(o);
                    if constexpr (WIDE)
#pragma unroll
                        for (int z = 0; z < 32; ++z) o[z] *= back;
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        *reinterpret_cast<uint4 *>(box_out + lane * 64 + ((z ^ (lane >> 1 & 3)) << 4)) =
                            make_uint4(pack2(o[8 * z] * inv, o[8 * z + 1] * inv, a.out_type),
                                       pack2(o[8 * z + 2] * inv, o[8 * z + 3] * inv, a.out_type),
                                       pack2(o[8 * z + 4] * inv, o[8 * z + 5] * inv, a.out_type),
                                       pack2(o[8 * z + 6] * inv, o[8 * z + 7] * inv, a.out_type));
                    __syncwarp();
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int r = 8 * z + (lane >> 2), ch = lane & 3, d = 32 * j + 8 * ch;
                        const uint4 v = *reinterpret_cast<const uint4 *>(box_out + r * 64 + ((ch ^ (r >> 1 & 3)) << 4));
                        const uint32_t g2 = t.first + 32 * w + r, t2 = g2 / static_cast<uint32_t>(a.group);
                        if (32 * w + r < t.rows && d < a.dim)
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (t.tok0 + t2) * a.out_token +
                                                       (head * a.group + (g2 - t2 * a.group)) * a.out_head + d) = v;
                    }
                    __syncwarp();
                }
                if (live && a.lse)
                    a.lse[static_cast<int64_t>(t.tok0 + tok) * a.lse_heads + hq] =
                        l == 0.0f ? -INFINITY : (m + log2f(l) - kShift) * kLn2;
            }
            tm_fence_before();
        }
    } else {
        regs_dec<other_regs(MODE)>();   // (a warpgroup changes its registers together)
        if constexpr (WIDE) {
            // -------------------------------------------------------- factors ahead
            // two units at a time: lane 16 j + 8 s + p has piece p of unit i + j, its keys' (s = 0) or values'
            int unit = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                Work item;
                ok = next_work(k, item);
                if (!ok || item.todo == 0) break;
                const bool holes = DOCS && (item.t.seq & kHoles);
                if (DOCS) item.t.seq &= ~kHoles;
                const Tile &t = item.t;
                const int first = t.lo / kChunkKeys + item.off;   // (tiles begin at pages)
                int top = 0;
                for (int i = 0; i < item.todo; i += 2) {
                    const bool mine = i + (lane >> 4) < item.todo;   // (the last may be alone)
                    const int kb = (first + i + (lane >> 4)) * kChunkKeys + 16 * (lane & 7);
                    // Only pieces that some row sees count: the others may hold any scale, and a tile that sees
                    // nothing has its unit behind the sequence's last page.
                    bool seen = mine && kb + 16 > t.from && kb < t.hi;
                    if (holes) {
                        for (int j = 0; j < min(2, item.todo - i); ++j) {
                            uint32_t all[kChunkKeys / 32];
                            seen_keys(a, t, (first + i + j) * kChunkKeys, all);
#pragma unroll
                            for (int z = 0; z < kChunkKeys / 32; ++z)
                                if ((lane >> 4) == j && (lane >> 1 & 3) == z) seen = (all[z] >> (16 * (lane & 1)) & 0xFFFFu) != 0;
                        }
                    }
                    float f = 0.0f;
                    if (seen)
                        f = a.factors[((static_cast<int64_t>(t.seq) * a.table_pages + first + i + (lane >> 4)) * a.kv_heads + item.head) * 16 +
                                      (lane & 15)];
                    if (__any_sync(0xffffffffu, f == -INFINITY)) {   // a piece that is not in the cache (whole warps: 1 % of the call)
                        if (f == -INFINITY) {
                            atomicOr(a.error, 4u);
                            f = 0.0f;
                        }
                    }
                    const int two = min(2, item.todo - i);
                    for (int z = 0; z < two && ok; ++z)
                        if (unit + z >= kUnitsAhead) ok = wait(sh.factors_empty[(unit + z) % kUnitsAhead], ((unit + z) / kUnitsAhead - 1) & 1);
                    if (!ok) break;
                    float most = (lane & 8) ? fabsf(f) : 0.0f;
#pragma unroll
                    for (int o = 8; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                    // the units' exponents (factors are at most 2^e), one after the other
                    const int e = max(-112, min(122, static_cast<int>(__float_as_uint(most) >> 23) - 126));
                    const int e0 = __shfl_sync(0xffffffffu, e, 0), e1 = two > 1 ? __shfl_sync(0xffffffffu, e, 16) : e0;
                    const int before = i == 0 ? e0 : top, top0 = max(before, e0);
                    top = max(top0, e1);
                    const int at = lane >> 4 ? top : top0, grown = lane >> 4 ? top - top0 : top0 - before;
                    const float keys = __shfl_xor_sync(0xffffffffu, f, 8);   // (to values: their keys')
                    UnitFactors &to = sh.factors[(unit + (lane >> 4)) % kUnitsAhead];
                    if (mine) {
                        if (lane & 8) {   // (below 2^-38 of the largest P is 0 in fp16; the sums, in fp32, still count)
                            float x = log2f(fabsf(f)) - static_cast<float>(at);
                            if (x < -60.0f) x = -60.0f;
                            if (keys != keys) x = keys;   // (a NaN among the factors of what is seen shows)
                            to.value[lane & 7] = x, to.undo[lane & 7] = ex2(-x);
                        } else {
                            to.key[lane & 7] = f;
                        }
                        if ((lane & 15) == 0) to.top = at, to.grown = grown;
                    }
                    __syncwarp();
                    if (mine && (lane & 15) == 0) mbar_arrive(smem_u32(&sh.factors_full[(unit + (lane >> 4)) % kUnitsAhead]));
                    unit += two;
                }
            }
        }
    }
    __syncwarp();
    tm_fence_before();
    __syncthreads();
    if (w == kMmaWarp) {
        if (*abort) {   // (else the softmax warps have seen the last products done)
            mma_commit(smem_u32(&sh.drained));
            (void)mbar_wait_bounded(smem_u32(&sh.drained), 0, kLandNs);
        }
        tm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512u) : "memory");
    }
}

struct ChunkLaunch {
    Args args;
    int device, sms;
    cudaStream_t stream;
};
cudaError_t launch_chunk_f16(const ChunkLaunch &l);
cudaError_t launch_chunk_bf16(const ChunkLaunch &l);
cudaError_t launch_chunk_wide(const ChunkLaunch &l);   // (a widened 8-bit cache)
// A call over an 8-bit cache: widened, then the kernel, in passes of as many cache heads
// (or sequences of one head) as kWidenMost bytes of scratch hold.  The host knows no length,
// only how wide the page table is.  Sixteen sequences of 256 tokens over 4096, 32 / 8 heads of
// 128, take 328 us in one pass, in 2 (a table of 65536 positions) 377, in 4 421; with 1 GiB
// they took 375 to 618, and the mma.sync kernel takes 2316.
constexpr int64_t kWidenMost = int64_t{4} << 30;
// What the library holds of it from call to call unless it is told otherwise: one such call's
// and its queries.  What is past that goes back to the system when the program synchronises,
// which costs 1.2 ms a GiB, and the next call 0.7 to take it again: with 1 GiB the above, its
// table of 32768, takes 2.8 ms between two synchronisations instead of 0.37.
constexpr int64_t kWidenKept = int64_t{5} << 30;
int64_t widened_bytes(const Args &a);   // of one cache head of one sequence
double widened_us(const Args &a, int64_t keys);
cudaError_t launch_widened(const ChunkLaunch &l);

}  // namespace attn
}  // namespace q4k
