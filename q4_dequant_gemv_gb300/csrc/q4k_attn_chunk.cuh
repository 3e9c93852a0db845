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
// 8-bit caches (CT = Q4K_I8, for codes of either type): the MMA's operands are fp16
// all the same, so codes become fp16 on their way into the stages.  Sixteen warps:
// warp 9 plans, units too (pages, seen keys, scales), some units ahead; warps 10 to 15
// take groups of 16 keys or values in turn, codes by 16-byte loads into registers one
// group ahead, converted, scaled and stored where TMA would have put them; at the start
// of a tile they turn the queries to fp16 over a power of two a row.  A unit's keys and
// values are over a power of two of its largest scale (128 of it at most), so that fp16
// holds them: the keys' joins the factor of the scores, the values' the exponents of P
// (relative to the largest so far, by which O is rescaled).  Per-column factors in the
// softmax instead would cost it 64 shared loads of 16 bytes a row and unit.
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

#include <type_traits>

#include "q4k_attn.cuh"
#include "q4k_codes.cuh"
#include "ptx.cuh"

namespace q4k {
namespace attn {

constexpr int kChunkRows = 256;              // query rows of a tile at most
constexpr int kChunkKeys = 128;              // keys of a unit
// two softmax warpgroups; MMA, key, value and idle warp, or MMA, planning and six converting warps
constexpr int chunk_threads(int type) { return eight(type) ? 512 : 384; }
constexpr int kMmaWarp = 8, kKeyWarp = 9, kValueWarp = 10;
constexpr int kStages = 4;
// 256 x 200 + 128 x 96 registers, within the 384 x 168 of the launch; 8 bits: 256 x 184 +
// 256 x 72, the 512 x 128 of the launch
constexpr int softmax_regs(int type) { return eight(type) ? 184 : 200; }
constexpr int other_regs(int type) { return eight(type) ? 72 : 96; }
constexpr int kPlanWarp = 9, kFirstConverter = 10, kConverters = 6;
constexpr int kUnits = 4;                    // units planned ahead

// A CTA's part of one tile, as the key warp found it.
struct Work {
    Tile t;
    int head, off, todo, last;   // units [off, off + todo) of the tile; the CTA that holds the tile's last unit
};

// (8 bits) A unit as the plan warp found it.
struct alignas(16) UnitInfo {
    float scale[2][kChunkKeys];              // of the keys and the values, over their powers of two; 0: not seen
    int page[8], slot[8];                    // of each piece of 16 keys
    uint32_t seen[kChunkKeys / 32];
    int head, kind;                          // kind 1: the first of a tile, 2: no more
    int exponent[2];                         // the powers of two
};
struct Planned {
    UnitInfo unit[kUnits];
    float row_scale[2][kChunkRows];          // of a tile's queries, two tiles
    unsigned long long full[kUnits], empty[kUnits];
};
struct NotPlanned {};

template <int CT, int DP>
struct ChunkShared {
    static constexpr int kHalf = 128 * 128;                    // bytes: 128 rows of 64 elements
    static constexpr int kTile = kHalf * (DP / 64);            // 128 rows of DP elements
    uint8_t q[2 * kTile];                                      // [dim / 64][256 rows][64]
    uint8_t kv[kStages * kTile];
    uint8_t out[8][32 * 64];                                   // a warp's rows on their way out, 32 columns at a time
    SplitShared<chunk_threads(CT)> plan;
    unsigned long long full[kStages], empty[kStages], s_full[2], p_ready[2][2], o_done[2], q_full, q_empty, edge, drained;
    unsigned long long work_full[2], work_empty[2];
    Work work[2];
    alignas(16) uint32_t seen[2][kChunkKeys / 32];   // (tiles with holes) of the key and the value warp
    typename std::conditional<eight(CT), Planned, NotPlanned>::type ahead;
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
    return CT == Q4K_BF16 ? 0.0f : 6.0f;
}

// (8 bits) Sixteen codes as fp16, times hi + lo (KEYS) or hi.
template <int CODES, bool KEYS>
__device__ __forceinline__ void convert16(const uint4 &raw, uint32_t hi, uint32_t lo, uint4 &a, uint4 &b)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        key_pairs<CODES>(w[i], r[2 * i], r[2 * i + 1]);
#pragma unroll
        for (int j = 2 * i; j < 2 * i + 2; ++j)   // (the product with hi is rounded once, lo's part before it)
            r[j] = KEYS ? hfma2_u32(r[j], hi, hmul2_u32(r[j], lo)) : hmul2_u32(r[j], hi);
    }
    a = make_uint4(r[0], r[1], r[2], r[3]), b = make_uint4(r[4], r[5], r[6], r[7]);
}

// MODE bit 0: capped scores, bit 1: distance bias, bit 2 (DOCS): a causal call with
// kv_start, whose tiles may have holes (its code in every instance cost 2048 tokens
// over 14336 positions 2 %).
template <int CT, int DP, int MODE>
__global__ void __launch_bounds__(chunk_threads(CT), 1)
    chunk_kernel(const __grid_constant__ CacheMaps maps, const __grid_constant__ CUtensorMap qmap, const Args a, const int box)
{
    using Sh = ChunkShared<CT, DP>;
    constexpr int kHalf = Sh::kHalf, kTile = Sh::kTile, ND = DP / 64, kOtherRegs = other_regs(CT);
    constexpr bool EIGHT = eight(CT);
    constexpr int FT = EIGHT ? Q4K_F16 : CT;   // the type of the products
    constexpr bool DOCS = MODE & 4;
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
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&sh.full[i]), EIGHT ? 8 : 1), mbar_init(smem_u32(&sh.empty[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.s_full[i]), 1);
            mbar_init(smem_u32(&sh.p_ready[i][0]), 128);
            mbar_init(smem_u32(&sh.p_ready[i][1]), 128);
            mbar_init(smem_u32(&sh.o_done[i]), 1);
            mbar_init(smem_u32(&sh.work_full[i]), 1);
            mbar_init(smem_u32(&sh.work_empty[i]), EIGHT ? 9 + kConverters : 10);   // the MMA, value (converting) and eight softmax warps
        }
        mbar_init(smem_u32(&sh.q_full), EIGHT ? kConverters : 1);
        if constexpr (EIGHT)
            for (int i = 0; i < kUnits; ++i) mbar_init(smem_u32(&sh.ahead.full[i]), 1), mbar_init(smem_u32(&sh.ahead.empty[i]), kConverters + 8);
        mbar_init(smem_u32(&sh.q_empty), 1);
        mbar_init(smem_u32(&sh.edge), 1);
        mbar_init(smem_u32(&sh.drained), 1);
        fence_barrier_init();
        sh.abort = 0;
    }
    if (!EIGHT && tid == 32) prefetch_tensormap(&maps.k), prefetch_tensormap(&maps.v), prefetch_tensormap(&qmap);
    tm_fence_before();
    pdl_launch_dependents();
    pdl_wait();   // (everything below may come from the kernel before)
    Split<kChunkKeys, chunk_threads(CT), kChunkKeys, DOCS> plan(a, sh.plan, tokens * a.group);   // synchronises the CTA
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

    if (EIGHT && w == kPlanWarp) {
        if constexpr (EIGHT) {
        // ------------------------------------------------------------ tiles and units ahead
        regs_dec<kOtherRegs>();
        int unit = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (k > 1 && !(ok = wait(sh.work_empty[k & 1], ((k >> 1) - 1) & 1))) break;
            Work item;
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
            const bool holes = DOCS && (item.t.seq & kHoles);
            if (DOCS) item.t.seq &= ~kHoles;
            const Tile &t = item.t;
            const int32_t *pages = a.page_table + static_cast<int64_t>(t.seq) * a.table_stride;
            const int kb0 = t.lo + item.off * kChunkKeys;
            // lane 8 j + p: piece p of unit first + j
            int ids = 0, slots = 0;
            auto look = [&](int first) {
                const int key = kb0 + first * kChunkKeys + 16 * lane;
                ids = slots = 0;
                if (first + (lane >> 3) < item.todo && key + 16 > t.from && key < t.hi) {
                    int e;
                    page_of(a, key, e, slots);
                    ids = pages[e];
                }
            };
            // lane: keys 4 lane .. of the unit, in piece lane / 4
            float sc[2][4];
            int page = 0, slot = 0;
            uint32_t seen[kChunkKeys / 32];
            auto fetch = [&](int i) {
                if ((i & 3) == 0) look(i);
                const int kb = kb0 + i * kChunkKeys;
                page = __shfl_sync(0xffffffffu, ids, 8 * (i & 3) + (lane >> 2));
                slot = __shfl_sync(0xffffffffu, slots, 8 * (i & 3) + (lane >> 2));
                if (holes) {
                    seen_keys(a, t, kb, seen);
                } else {
#pragma unroll
                    for (int z = 0; z < kChunkKeys / 32; ++z) seen[z] = span(t.from - kb - 32 * z, t.hi - kb - 32 * z);
                }
                // a piece that some row sees must be in the cache
                uint32_t mine = 0;   // the word of this lane's keys
#pragma unroll
                for (int z = 0; z < kChunkKeys / 32; ++z) mine = (lane >> 3) == z ? seen[z] : mine;
                const bool bad = (mine >> (16 * (lane >> 2 & 1)) & 0xFFFFu) && (page < 0 || page >= a.pages);
                const uint32_t lost = __ballot_sync(0xffffffffu, bad);
                if (lost) {
                    if (lane == 0) atomicOr(a.error, 4u);
#pragma unroll
                    for (int z = 0; z < kChunkKeys / 32; ++z)
                        seen[z] &= ~((lost >> 8 * z & 1 ? 0xFFFFu : 0u) | (lost >> (8 * z + 4) & 1 ? 0xFFFF0000u : 0u));
#pragma unroll
                    for (int z = 0; z < kChunkKeys / 32; ++z) mine = (lane >> 3) == z ? seen[z] : mine;
                }
                const float *kp = a.ks + page * a.ks_page + item.head * a.ks_head, *vp = a.vs + page * a.vs_page + item.head * a.vs_head;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int s = slot + 4 * (lane & 3) + z;
                    const bool live = mine >> (4 * (lane & 7) + z) & 1;
                    sc[0][z] = live ? kp[(s >> a.block_shift) * a.ks_block] : 0.0f;
                    sc[1][z] = live ? vp[(s >> a.block_shift) * a.vs_block] : 0.0f;
                }
            };
            if (item.todo > 0) fetch(0);
            for (int i = 0; i < item.todo + (item.todo == 0 ? 1 : 0); ++i, ++unit) {
                UnitInfo &info = sh.ahead.unit[unit % kUnits];
                if (unit >= kUnits && !(ok = wait(sh.ahead.empty[unit % kUnits], (unit / kUnits - 1) & 1))) break;
                if (item.todo > 0) {
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        const float most = fmaxf(fmaxf(fabsf(sc[side][0]), fabsf(sc[side][1])), fmaxf(fabsf(sc[side][2]), fabsf(sc[side][3])));
                        const int e = static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(most)) >> 23) - 133;
                        const int x = max(-120, min(115, e));   // the largest to [64, 128)
                        const float f = two_to(-x);
                        *reinterpret_cast<float4 *>(&info.scale[side][4 * lane]) =
                            make_float4(sc[side][0] * f, sc[side][1] * f, sc[side][2] * f, sc[side][3] * f);
                        if (lane == 0) info.exponent[side] = x;
                    }
                    if ((lane & 3) == 0) info.page[lane >> 2] = page, info.slot[lane >> 2] = slot;
                    if (lane == 0) {
#pragma unroll
                        for (int z = 0; z < kChunkKeys / 32; ++z) info.seen[z] = seen[z];
                    }
                }
                if (lane == 0) info.head = item.head, info.kind = item.todo == 0 ? 2 : i == 0 ? 1 : 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.ahead.full[unit % kUnits]));
                if (i + 1 < item.todo) fetch(i + 1);
            }
            if (item.todo == 0) break;
        }
        }
    } else if (EIGHT && w >= kFirstConverter) {
        if constexpr (EIGHT) {
        // ------------------------------------------------------------ codes to fp16
        regs_dec<kOtherRegs>();
        const int cw = w - kFirstConverter;
        // a group's loads: this lane's chunk of 16 codes of rows row0 + ROWS j; eight lanes store
        // four chunks of two neighbouring rows, which the swizzle puts into eight places
        constexpr int LOADS = DP / 32, ROWS = 16 / LOADS;
        const int ch = DP == 128 ? (lane & 3) + (lane >> 1 & 4) : lane & 3;
        const int row0 = DP == 128 ? (lane >> 2 & 1) + (lane >> 3 & 2) : lane >> 2;
        const bool inside = 16 * ch < a.dim;
        // a group's rows: where they are, which of them some row of the tile sees
        const uint8_t *from = nullptr;
        int64_t step = 0;
        uint32_t seen = 0;
        auto aim = [&](const UnitInfo &info, int part) {
            const int piece = part & 7;
            const bool values = part >= 8;
            seen = inside ? info.seen[piece >> 1] >> (16 * (piece & 1) + row0) : 0u;
            step = values ? a.v_slot : a.k_slot;
            from = static_cast<const uint8_t *>(values ? a.v : a.k) + info.page[piece] * (values ? a.v_page : a.k_page) +
                   info.head * (values ? a.v_head : a.k_head) + (info.slot[piece] + row0) * step + 16 * ch;
            step *= ROWS;
        };
        auto load = [&](int j) {
            uint4 r = make_uint4(0, 0, 0, 0);
            if (seen >> (ROWS * j) & 1) r = __ldg(reinterpret_cast<const uint4 *>(from + j * step));
            return r;
        };
        // the tile's queries: rows of 16 (8) lanes, in fp16 over a power of two
        auto queries = [&](int k) -> bool {
            if (!wait(sh.work_full[k & 1], (k >> 1) & 1)) return false;
            const Work &item = sh.work[k & 1];
            const int tok0 = item.t.tok0, first = item.t.first, rows = item.t.rows, hq0 = item.head * a.group;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.work_empty[k & 1]));
            if (k > 0 && !wait(sh.q_empty, (k - 1) & 1)) return false;
            constexpr int LANES = DP / 8, PER = 32 / LANES, DEEP = 4;
            const int c = lane % LANES;
            const uint16_t *q = static_cast<const uint16_t *>(a.q);
#pragma unroll 1
            for (int r0 = cw * PER; r0 < kChunkRows; r0 += DEEP * kConverters * PER) {
                uint4 raw[DEEP];
#pragma unroll
                for (int j = 0; j < DEEP; ++j) {
                    const int r = r0 + j * kConverters * PER + lane / LANES;
                    raw[j] = make_uint4(0, 0, 0, 0);
                    if (r < rows && 8 * c < a.dim) {
                        const uint32_t x = first + r, tok = x / static_cast<uint32_t>(a.group);
                        raw[j] = __ldg(reinterpret_cast<const uint4 *>(q + (tok0 + tok) * a.q_token + (hq0 + static_cast<int>(x - tok * a.group)) * a.q_head + 8 * c));
                    }
                }
#pragma unroll
                for (int j = 0; j < DEEP; ++j) {
                    const int r = r0 + j * kConverters * PER + lane / LANES;
                    const uint32_t w4[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
                    float mx = 0.0f;
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float2 f = unpack2(w4[z], a.q_type);
                        mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
#pragma unroll
                    for (int o = LANES / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const int ex = static_cast<int>(__float_as_uint(mx) >> 23);
                    const int e = ex != 0 && ex != 255 ? max(-126, min(126, 141 - ex)) : 0;   // max|q| to [2^14, 2^15)
                    const float up = two_to(e);
                    uint32_t h[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float2 f = unpack2(w4[z], a.q_type);
                        h[z] = pack2(f.x * up, f.y * up, Q4K_F16);
                    }
                    if (r < kChunkRows) {
                        *reinterpret_cast<uint4 *>(sh.q + (c >> 3) * 2 * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                            make_uint4(h[0], h[1], h[2], h[3]);
                        if (c == 0) sh.ahead.row_scale[k & 1][r] = two_to(-e);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.q_full));
            return true;
        };
        uint4 raw[LOADS];
        int tile = 0;
        bool ok = true, more = true;
        // the first of this warp's groups of a unit: whether there is one, then whether its tile begins there
        auto begin = [&](int un) -> bool {
            if (!wait(sh.ahead.full[un % kUnits], (un / kUnits) & 1)) return ok = false;
            return more = sh.ahead.unit[un % kUnits].kind != 2;
        };
        // group g: unit g / 16; its keys' pieces, then its values'
        int g = cw;
        (void)begin(0);
        while (ok && more) {
            const int un = g >> 4, part = g & 15;
            const UnitInfo &info = sh.ahead.unit[un % kUnits];
            if (part < kConverters && info.kind == 1) {   // a tile begins: its queries first
                if (!(ok = queries(tile++))) break;
                aim(info, part);
#pragma unroll
                for (int j = 0; j < LOADS; ++j) raw[j] = load(j);
            }
            const bool values = part >= 8;
            const int stage = 2 * (un & 1) + (values ? 1 : 0), piece = part & 7;
            const int next = g + kConverters;
            const bool last = (next >> 4) != un;   // of this unit's groups
            // the next group's codes are on their way while this one's are converted (but for a new tile's)
            bool ahead = !last;
            if (last && begin(next >> 4)) ahead = sh.ahead.unit[(next >> 4) % kUnits].kind == 0;
            if (!ok || (un > 1 && !(ok = wait(sh.empty[stage], ((un >> 1) - 1) & 1)))) break;
            seen = 0;
            if (ahead) aim(sh.ahead.unit[(next >> 4) % kUnits], next & 15);
            uint8_t *dst = sh.kv + stage * kTile + (ch >> 2) * kHalf;
            const float *scales = &info.scale[values][16 * piece + row0];
            // (one straight line for each kind, so that the rows' chains run side by side)
            auto convert = [&](auto codes, auto keys) {
                uint32_t hi[LOADS], lo[LOADS];
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    const float s = scales[ROWS * j];
                    const __half h = __float2half_rn(s);
                    hi[j] = __half_as_ushort(h) * 0x10001u;
                    lo[j] = decltype(keys)::value ? __half_as_ushort(__float2half_rn(s - __half2float(h))) * 0x10001u : 0u;
                }
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    uint4 x, y;
                    convert16<decltype(codes)::value, decltype(keys)::value>(raw[j], hi[j], lo[j], x, y);
                    raw[j] = load(j);
                    // (rows of a lane are 8 apart, or 4: the swizzle's place changes with bit 2)
                    const int at = (16 * piece + row0 + ROWS * j) * 128 + ((2 * (ch & 3) ^ ((row0 + ROWS * j) & 7)) << 4);
                    *reinterpret_cast<uint4 *>(dst + at) = x;
                    *reinterpret_cast<uint4 *>(dst + (at ^ 16)) = y;
                }
            };
            if (a.codes == Q4K_I8) {
                if (values) convert(std::integral_constant<int, Q4K_I8>{}, std::false_type{});
                else convert(std::integral_constant<int, Q4K_I8>{}, std::true_type{});
            } else {
                if (values) convert(std::integral_constant<int, Q4K_E4M3>{}, std::false_type{});
                else convert(std::integral_constant<int, Q4K_E4M3>{}, std::true_type{});
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (!(a.stall && g == 0)) mbar_arrive(smem_u32(&sh.full[stage]));
                if (last) mbar_arrive(smem_u32(&sh.ahead.empty[un % kUnits]));
            }
            g = next;
        }
        }
    } else if (!EIGHT && (w == kKeyWarp || w == kValueWarp)) {
        // ------------------------------------------------------------ loads
        regs_dec<kOtherRegs>();
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
                    page = pages[e];
                    if (page < 0 || page >= a.pages) {
                        atomicOr(a.error, 4u);
                        live = false;
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
        regs_dec<kOtherRegs>();
        constexpr uint32_t id_s = chunk_idesc<FT>(kChunkKeys, false), id_o = chunk_idesc<FT>(DP, true);
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
        regs_inc<softmax_regs(CT)>();
        const int h = w >> 2, row = tid;                // row of the tile: half h, TMEM lane tid % 128
        const uint32_t lane_base = static_cast<uint32_t>(w & 3) << 21;   // 32 (w % 4) lanes, in bits 16..
        const uint32_t ts = tm + lane_base + 128 * h, to = tm + lane_base + 256 + 128 * h;
        uint32_t steps = 0, done = 0;
        int unit = 0;                   // (8 bits) units of this CTA so far
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
                if constexpr (EIGHT) {   // (the tile is not this warp's, but its phases are)
                    ok = wait(sh.q_full, k & 1);
                    for (int i = 0; i < todo && ok; ++i, ++unit) {
                        ok = wait(sh.ahead.full[unit % kUnits], (unit / kUnits) & 1);
                        if (ok && lane == 0) mbar_arrive(smem_u32(&sh.ahead.empty[unit % kUnits]));
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
            float cq = c;                    // (8 bits) with the power of two of the row's queries
            int top = 0;                     // (8 bits) O is over 2^top
            if constexpr (EIGHT) {
                ok = wait(sh.q_full, k & 1);
                if (!ok) break;
                cq = c * sh.ahead.row_scale[k & 1][row];
            }
            for (int i = 0; i < todo; ++i) {
                const int kb = t.lo + (off + i) * kChunkKeys;
                ok = wait(sh.s_full[h], steps & 1);
                if (!ok) break;
                ++steps;
                tm_fence_after();
                float cu = c;
                int low = 0;       // (8 bits) the unit's values are over 2^(top + low), low <= 0
                int grown = 0;     // (8 bits) by which the unit raises top
                if constexpr (EIGHT) {
                    const int un = unit++ % kUnits;
                    ok = wait(sh.ahead.full[un], ((unit - 1) / kUnits) & 1);
                    if (!ok) break;
                    // (below 1e-30 a score is nothing, and one masked out has to stay -inf)
                    cu = fminf(fmaxf(cq * two_to(sh.ahead.unit[un].exponent[0]), 1e-30f), 3e38f);
                    const int x = sh.ahead.unit[un].exponent[1];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.ahead.empty[un]));
                    if (i == 0) top = x;
                    grown = max(x - top, 0);
                    top += grown;
                    low = max(x - top, -100);
                }
                float s[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tm_ld32(ts + 32 * q, s[q]);
                tm_wait_ld32(s[0]);
#pragma unroll
                for (int q = 1; q < 4; ++q) tm_here32(s[q]);
                float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float *v = s[q];
                    if (MODE & 1) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = a.softcap * kLog2e * (1.0f - 2.0f * rcp(ex2(2.0f * kLog2e * (v[j] * cu)) + 1.0f));
                    }
                    if (MODE & 2) {
                        const float d0 = static_cast<float>(rel - kb - 32 * q);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = fmaf(-slope, fabsf(d0 - static_cast<float>(j)), (MODE & 1) ? v[j] : v[j] * cu);
                    }
                    if (kb < in_lo || kb + kChunkKeys > in_hi) {
                        const int a0 = lo - kb - 32 * q, a1 = hi - kb - 32 * q;
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = j >= a0 && j < a1 ? v[j] : -INFINITY;
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
#pragma unroll
                        for (int z = 0; z < 4; ++z) x[z] = max3(x[z], v[j + 2 * z], v[j + 2 * z + 1]);
                    }
                }
                const float mul = (MODE & 3) ? 1.0f : cu;
                const float mx = fmaxf(max3(x[0], x[1], x[2]), x[3]) * mul;
                float f = 1.0f;
                if (mx > m + kLazy || m == -INFINITY) {
                    // (m = mx = -inf: everything masked so far, l and O are zero)
                    f = mx == m ? 1.0f : ex2(m - mx);
                    m = mx;
                }
                if (i > 0 && (__any_sync(0xffffffffu, f != 1.0f) || (EIGHT && grown))) {
                    l *= f;
                    if constexpr (EIGHT) f *= two_to(max(-grown, -126));
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
                const float base = (m == -INFINITY ? 0.0f : m - kShift) - static_cast<float>(low);
                const uint64_t mul2 = pair(mul, mul), base2 = pair(-base, -base);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t p[16];
#pragma unroll
                    for (int z = 0; z < 16; ++z) {
                        float e0, e1;
                        unpair(fma2(pair(s[q][2 * z], s[q][2 * z + 1]), mul2, base2), e0, e1);
                        e0 = ex2(e0), e1 = ex2(e1);
                        sum[z & 1] = add2(sum[z & 1], pair(e0, e1));
                        p[z] = pack2(e0, e1, FT);
                    }
                    tm_st16(ts + 16 * q, p);
                    if (q & 1) {   // 64 keys of P: the products can start on them
                        tm_wait_st();
                        tm_fence_before();
                        mbar_arrive(smem_u32(&sh.p_ready[h][q >> 1]));
                    }
                }
                float l0, l1;
                unpair(add2(sum[0], sum[1]), l0, l1);
                l += EIGHT ? (l0 + l1) * two_to(-low) : l0 + l1;
            }
            if (!ok) break;
            const float back = EIGHT ? two_to(top) : 1.0f;   // O's power of two

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
                    if constexpr (EIGHT)
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
                    if constexpr (EIGHT)
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
                    a.lse[static_cast<int64_t>(t.tok0 + tok) * a.heads + hq] =
                        l == 0.0f ? -INFINITY : (m + log2f(l) - kShift) * kLn2;
            }
            tm_fence_before();
        }
    } else {
        regs_dec<kOtherRegs>();   // (a warpgroup changes its registers together)
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
cudaError_t launch_chunk_8(const ChunkLaunch &l);

}  // namespace attn
}  // namespace q4k
