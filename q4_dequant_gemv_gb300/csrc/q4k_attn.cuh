// q4k_attn.cuh -- what the attention kernels share: the arguments, the split of
// a call's work over the CTAs, and the join of split rows.
//
// A sequence's query rows for one cache head are its (token, head of the group)
// pairs, row r = token r / G, head r % G of the group (G = query heads per cache
// head).  A tile is R consecutive rows of one sequence and one cache head; its
// work is counted in units of U keys over the keys that any of its rows sees.
// Lengths live on the device, so every CTA works the split out by itself: it
// sums the units of all tiles (a prefix over the call, identical in every CTA)
// and takes an equal, contiguous share of them, wherever that begins or ends
// inside a tile.  The load is therefore even for ragged lengths, causal tiles
// and one long sequence alike, with no host knowledge of lengths.  Rows of a
// tile that several CTAs hold meet in scratch memory, where a second kernel, its
// launch hidden under the first, adds the partial results in the order of the
// keys, so the same inputs give the same bits.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "../../include/q4k.h"

namespace q4k {
namespace attn {

// Packed pairs of a 16-bit type (Q4K_F16 or Q4K_BF16), low half first.
__device__ __forceinline__ float2 unpack2(uint32_t v, int type)
{
    if (type == Q4K_F16) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&v);
        return __half22float2(h);
    }
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int type)
{
    uint32_t r;
    if (type == Q4K_F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

struct Args {
    const void *q, *k, *v;
    void *out;
    float *lse;
    int64_t q_token, q_head, out_token, out_head;        // strides in elements
    int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
    int64_t table_stride;
    int page_size;
    const int32_t *page_table, *seq_start, *kv_len, *prefix_len, *kv_start;
    const float *slopes;
    int capacity;          // cached positions a page table row can hold
    int window;            // 0: none
    int page_shift;        // page_size = 1 << page_shift, or -1
    float scale, softcap;
    int pages, batch, tokens, heads, kv_heads, group, dim;
    int q_type, out_type, causal;
    int slots;             // upper bound of the tiles per cache head
    int cluster;           // few-rows kernel: CTAs of a cluster that share a tile; 0: the split over all CTAs
    float *part;           // partial results: two slots per CTA
    struct Joint *joint;   // the split tile that starts in each CTA's share
    unsigned int *error;   // the sticky error word
    uint64_t wait_ns;      // bound of each wait
    int stall;             // (tests) the first copy of a CTA is awaited for 16 bytes too many
    bool pdl;              // launched as a programmatic dependent

    // Tiles of the call may have keys that no row sees between some that one sees.
    __host__ __device__ bool docs() const { return kv_start && causal; }
};

// A split tile: its rows, and the CTAs c0 .. c1 that hold its parts.  The first of
// them has its part in its second slot (the tile begins in its share), the others
// in their first slots.  A slot is [dim / 4][R] quads of O, R maxima (log2), R sums.
struct alignas(32) Joint {
    int tok0, first, rows, head, c0, c1;
};

__device__ __forceinline__ int64_t part_slot(int cta, bool begins) { return 2 * static_cast<int64_t>(cta) + (begins ? 1 : 0); }

constexpr int kHoles = 1 << 30;

// How long a kernel that winds down waits for a copy or product in flight, whatever
// limit the call gave its waits: they end in microseconds, and shared and tensor
// memory are not given up before.
constexpr uint64_t kLandNs = 20000000;

// One tile: the rows, their token range and the keys that any of them sees.
struct Tile {
    int seq;                   // (+ kHoles: between `from` and `hi` there may be keys that no row sees)
    int first, rows;           // first row in the sequence, number of rows (0: nothing to do)
    int tok0;                  // first token row of the sequence in the call
    int pos0;                  // position of the sequence's first new token
    int len;                   // cached positions (clamped to the page table)
    int from, hi;              // keys [from, hi) that some row sees
    int lo;                    // `from` rounded down to a multiple of ALIGN: where unit 0 starts
    int units;
};

struct Range {
    int lo, hi;
};

// Keys that the new token in row `tok` of the call, at position pos, sees.
// (Lengths leave room above positions, so nothing here overflows.)
__device__ __forceinline__ Range token_range(const Args &a, int seq, int pos, int tok, int len)
{
    Range r{0, len};
    if (a.causal) {
        int h = pos + 1;
        if (a.prefix_len) h = max(h, a.prefix_len[seq]);
        r.hi = min(h, len);
    }
    if (a.window) r.lo = max(r.lo, pos + 1 - a.window);
    if (a.kv_start) r.lo = max(r.lo, a.kv_start[tok]);
    r.hi = max(r.hi, 0);
    r.lo = min(r.lo, r.hi);
    return r;
}

// Bits [lo, hi) of a word, cut to it.
__device__ __forceinline__ uint32_t span(int lo, int hi)
{
    lo = max(lo, 0), hi = min(hi, 32);
    return hi > lo ? (0xFFFFFFFFu >> (32 - (hi - lo))) << lo : 0u;
}

// The 32 WORDS keys from kb on that some row of a tile sees, a bit each; whole warps.
template <int WORDS>
__device__ __forceinline__ void seen_keys(const Args &a, const Tile &t, int kb, uint32_t (&seen)[WORDS])
{
    const int last = (t.first + t.rows - 1) / a.group;
#pragma unroll
    for (int w = 0; w < WORDS; ++w) seen[w] = 0;
#pragma unroll 1
    for (int i = t.first / a.group + static_cast<int>(threadIdx.x & 31); i <= last; i += 32) {
        const Range r = token_range(a, t.seq, t.pos0 + i, t.tok0 + i, t.len);
#pragma unroll
        for (int w = 0; w < WORDS; ++w) seen[w] |= span(r.lo - kb - 32 * w, r.hi - kb - 32 * w);
    }
#pragma unroll
    for (int w = 0; w < WORDS; ++w) seen[w] = __reduce_or_sync(0xffffffffu, seen[w]);
}

// The split of the call's work, one copy per CTA in shared memory.
// R (rows of a tile) is given at run time; ALIGN: where units start (a power of two);
// DOCS: tiles are marked where they may have holes (causal calls with kv_start).
template <int THREADS>
struct SplitShared {
    static constexpr int kSeqs = 512;        // sequence starts held in shared memory
    uint32_t prefix[THREADS];                // units up to the end of each stripe of tile slots
    int start[kSeqs + 1], len[kSeqs];
    uint32_t warp[THREADS / 32];
    Tile first;                              // the tile of `hand_out`
    int offset;
};

template <int U, int THREADS, int ALIGN, bool DOCS>
struct Split {
    using Shared = SplitShared<THREADS>;
    static constexpr int kSeqs = Shared::kSeqs;

    const Args &a;
    Shared &sh;
    const int R;
    int stripe;             // slots of a prefix entry
    Tile mine;              // the slot of this thread where an entry is one slot (without kv_start)
    uint32_t before;        // units before this thread's entry
    uint32_t per_head;      // units of one cache head

    __device__ __forceinline__ int start_of(int b) const
    {
        const int s = a.batch <= kSeqs ? sh.start[b] : a.seq_start[b];
        return min(max(s, 0), a.tokens);
    }
    // Tile slots: slot b < batch is sequence b's first tile; its others take the
    // slots from batch + extra(b) on, which has room for them whatever the lengths.
    __device__ __forceinline__ int extra(int b) const
    {
        return static_cast<int>(static_cast<uint32_t>(start_of(b)) * static_cast<uint32_t>(a.group) / static_cast<uint32_t>(R));
    }

    // The tile of a slot.  WARP: by a whole warp, reporting lengths that do not fit
    // the page table; else by one thread, for calls without kv_start.
    template <bool WARP>
    __device__ __forceinline__ Tile tile(int slot) const
    {
        Tile t{};
        int b = slot, j = 0;
        if (slot >= a.batch) {
            const int x = slot - a.batch;
            int e = a.batch - 1;
            b = 0;
            while (b < e) {   // the last sequence with extra(b) <= x
                const int m = (b + e + 1) >> 1;
                if (extra(m) <= x) b = m; else e = m - 1;
            }
            j = x - extra(b) + 1;
        }
        const int s0 = start_of(b), n = start_of(b + 1) - s0, all = n * a.group;
        const int raw = a.batch <= kSeqs ? sh.len[b] : a.kv_len[b];
        t.seq = b, t.tok0 = s0;
        if (n <= 0 || j < 0 || j > (all - 1) / R) return t;
        t.first = j * R;
        t.rows = min(R, all - t.first);
        t.len = min(max(raw, 0), a.capacity);
        if (WARP && (raw < 0 || raw > a.capacity)) atomicOr(a.error, 4u);
        t.pos0 = max(raw, -1) - n;
        // its tokens (all of them where one tile holds the sequence)
        int i0 = 0, i1 = n - 1;
        if (all > R) i0 = t.first / a.group, i1 = (t.first + t.rows - 1) / a.group;
        const Range last = token_range(a, b, t.pos0 + i1, s0 + i1, t.len);
        int lo = last.hi;
        if (WARP && a.kv_start) {
            bool away = false;   // a token does not see its own position
#pragma unroll 4
            for (int i = i0 + static_cast<int>(threadIdx.x & 31); i <= i1; i += 32) {
                const Range r = token_range(a, b, t.pos0 + i, s0 + i, t.len);
                if (r.hi > r.lo) lo = min(lo, r.lo);
                if constexpr (DOCS) away |= r.lo > t.pos0 + i;
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            if (lo >= last.hi) lo = (lo + ALIGN - 1) & ~(ALIGN - 1);   // sees nothing: no key is looked up
            // Where every token sees its own position the ranges of consecutive ones meet,
            // and where the mask is not causal all end together: no holes.
            if constexpr (DOCS)
                if (__any_sync(0xffffffffu, away)) t.seq |= kHoles;
        } else {
            lo = min(lo, token_range(a, b, t.pos0 + i0, s0 + i0, t.len).lo);
        }
        t.hi = last.hi;
        t.from = lo;
        t.lo = lo & ~(ALIGN - 1);
        t.units = t.hi > t.lo ? (t.hi - t.lo + U - 1) / U : 1;   // a tile that sees nothing still writes its zeros
        return t;
    }

    // Sequence starts and lengths; all threads of the CTA.
    __device__ __forceinline__ Split(const Args &args, Shared &shared, int rows) : a(args), sh(shared), R(rows)
    {
        const int tid = threadIdx.x;
        for (int i = tid; i <= a.batch; i += THREADS) {
            // (all three on their way before any is looked at)
            const int s = a.seq_start[i], before = i > 0 ? a.seq_start[i - 1] : 0, len = i < a.batch ? a.kv_len[i] : 0;
            if (a.batch <= kSeqs) {
                sh.start[i] = s;
                if (i < a.batch) sh.len[i] = len;
            }
            if (s < before || s < 0 || s > a.tokens) atomicOr(a.error, 4u);
        }
        __syncthreads();
    }

    // The prefix over all tiles; all threads of the CTA.
    __device__ __forceinline__ void scan()
    {
        const int tid = threadIdx.x;
        stripe = (a.slots + THREADS - 1) / THREADS;
        uint32_t units = 0;
        if (a.kv_start) {   // a warp per entry: its lanes share a tile's tokens
            const int entries = (a.slots + stripe - 1) / stripe;
            for (int e = tid >> 5; e < entries; e += THREADS / 32) {
                uint32_t n = 0;
                for (int s = e * stripe; s < min((e + 1) * stripe, a.slots); ++s) n += tile<true>(s).units;
                if ((tid & 31) == 0) sh.prefix[e] = n;
            }
            __syncthreads();
            if (tid < entries) units = sh.prefix[tid];
        } else {
            for (int s = tid * stripe; s < min((tid + 1) * stripe, a.slots); ++s) {
                mine = tile<false>(s);
                units += mine.units;
            }
        }
        uint32_t incl = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if ((tid & 31) >= o) incl += v;
        }
        if ((tid & 31) == 31) sh.warp[tid >> 5] = incl;
        __syncthreads();
        uint32_t base = 0, total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < (tid >> 5)) base += sh.warp[w];
            total += sh.warp[w];
        }
        before = base + incl - units;
        sh.prefix[tid] = base + incl;
        per_head = total;
    }

    // Where each entry is one slot, the thread that holds unit r leaves its tile in
    // `first`; all threads of the CTA (it also completes the prefix).  False:
    // `locate` has to find it.
    __device__ __forceinline__ bool hand_out(uint32_t r)
    {
        const bool known = stripe == 1 && !a.kv_start;
        if (known && r >= before && r < sh.prefix[threadIdx.x]) {
            sh.first = mine, sh.offset = static_cast<int>(r - before);
            const int len = a.batch <= kSeqs ? sh.len[mine.seq] : a.kv_len[mine.seq];
            if (len < 0 || len > a.capacity) atomicOr(a.error, 4u);
        }
        __syncthreads();
        return known;
    }

    // The tile that holds unit r (< per_head) of a cache head, and r's place in it; whole warps.
    __device__ __forceinline__ Tile locate(uint32_t r, int &offset) const
    {
        int lo = 0, hi = THREADS - 1;
        while (lo < hi) {
            const int m = (lo + hi) >> 1;
            if (sh.prefix[m] > r) hi = m; else lo = m + 1;
        }
        uint32_t at = lo ? sh.prefix[lo - 1] : 0;
        for (int s = lo * stripe;; ++s) {
            const Tile t = tile<true>(s);
            if (at + t.units > r || s + 1 >= a.slots) {
                offset = static_cast<int>(r - at);
                return t;
            }
            at += t.units;
        }
    }
};

// a / b for non-negative a, b > 0 (a 64-bit division takes ten times a 32-bit one).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// A unit's place within its cache head.
__device__ __forceinline__ uint32_t per_head_rest(int64_t unit, uint32_t per_head)
{
    return per_head ? static_cast<uint32_t>(unit - quotient(unit, per_head) * per_head) : 0u;
}

// How many of `grid` CTAs share `total` units: at least two units each (a part
// costs the join more than a unit saves).
__device__ __forceinline__ int sharers(int64_t total, int grid) { return static_cast<int>(min(static_cast<int64_t>(grid), (total + 1) / 2)); }

// A CTA's share [begin, end) of `total` units over n CTAs, and the CTA that
// holds a unit.
__device__ __forceinline__ int64_t share_begin(int64_t total, int n, int c) { return quotient(total * c, n); }
__device__ __forceinline__ int share_owner(int64_t total, int n, int64_t unit)
{
    return static_cast<int>(quotient((unit + 1) * n - 1, total));
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Weight of a partial result with maximum m in a sum with maximum mx.  One that
// saw nothing (m = -inf) holds zeros, or a NaN to pass on (fmaxf drops NaN from
// the maxima, the sums carry it).
__device__ __forceinline__ float weight(float m, float mx) { return m == -INFINITY ? 1.0f : ex2(m - mx); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Four consecutive outputs of a row.
__device__ __forceinline__ void store4(void *out, int type, int64_t i, float4 v)
{
    if (type == Q4K_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + i) = v;
    } else {
        uint2 w;
        w.x = pack2(v.x, v.y, type);
        w.y = pack2(v.z, v.w, type);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + i) = w;
    }
}

// Four outputs from d on of query head hq in row tok of the call: v / ls; and the
// row's lse with d = 0.  m and ls as the kernels keep them: log2 domain, ls
// carrying 2^shift.
__device__ __forceinline__ void finish_row(const Args &a, int64_t tok, int hq, int d, float4 v, float m, float ls, float shift)
{
    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    store4(a.out, a.out_type, tok * a.out_token + hq * a.out_head + d,
           make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    if (a.lse && d == 0) a.lse[tok * a.heads + hq] = ls == 0.0f ? -INFINITY : (m + log2f(ls) - shift) * kLn2;
}

// Page (index into the sequence's table) and slot of a cached position.
__device__ __forceinline__ void page_of(const Args &a, int key, int &entry, int &slot)
{
    entry = a.page_shift >= 0 ? key >> a.page_shift
                              : static_cast<int>(static_cast<uint32_t>(key) / static_cast<uint32_t>(a.page_size));
    slot = key - entry * a.page_size;
}

// The cache as two 4-D tensors [page][head][slot][d], and a box of one cache
// head of a page: some slots by 64 elements, 128-byte swizzle.
struct CacheMaps {
    CUtensorMap k, v;
};

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int d, int slot, int head, int page,
                                         uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(d), "r"(slot), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

// Host: what a device needs once (a kernel's limits, a pool): `make` runs under a
// lock until it has succeeded.  A failure goes to its caller; the next call tries again.
constexpr int kDevices = 64;
struct OncePerDevice {
    std::atomic<uint64_t> made{0};
    std::mutex lock;

    template <class Make>
    cudaError_t operator()(int dev, Make make)
    {
        if (made.load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
        const std::lock_guard<std::mutex> hold(lock);
        if (made.load(std::memory_order_relaxed) >> dev & 1) return cudaSuccess;
        const cudaError_t e = make();
        if (e == cudaSuccess) made.fetch_or(uint64_t{1} << dev, std::memory_order_release);
        return e;
    }
};

// Host: scratch of `grid` CTAs, the first kernel by `launch(args)`, the join of the
// tiles that it left split; R rows and `width` columns a slot.
constexpr int kJoinThreads = 256, kJoinRows = 32;   // of a CTA of the join at most
constexpr int kMaxParts = 184;   // CTAs of a split call at most (the join's statistics: 47 KB)
cudaError_t take_scratch(int dev, void **p, size_t bytes, cudaStream_t stream);   // freed with cudaFreeAsync
cudaError_t launch_join(const Args &a, int grid, int R, int width, float shift, cudaStream_t stream);

template <class Launch>
cudaError_t launch_split(Args &a, int dev, int grid, int R, int width, float shift, cudaStream_t stream, Launch launch)
{
    const size_t head = (grid * sizeof(Joint) + 255) / 256 * 256;
    void *scratch = nullptr;
    cudaError_t e = take_scratch(dev, &scratch, head + static_cast<size_t>(grid) * 2 * R * (width + 2) * sizeof(float), stream);
    if (e != cudaSuccess) return e;
    a.joint = static_cast<Joint *>(scratch);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(scratch) + head);
    e = launch(a);
    if (e == cudaSuccess) e = launch_join(a, grid, R, width, shift, stream);
    const cudaError_t f = cudaFreeAsync(scratch, stream);
    return e == cudaSuccess ? f : e;
}

// Host: the launch attributes of a first kernel: clusters of `cluster` CTAs (0:
// none), a programmatic dependent of the kernel before.
struct Attributes {
    cudaLaunchAttribute at[2];
    Attributes(cudaLaunchConfig_t *cfg, int cluster, bool pdl)
    {
        cfg->attrs = at;
        cfg->numAttrs = 0;
        if (cluster > 0) {
            cudaLaunchAttribute &c = at[cfg->numAttrs++];
            c.id = cudaLaunchAttributeClusterDimension;
            c.val.clusterDim.x = cluster, c.val.clusterDim.y = 1, c.val.clusterDim.z = 1;
        }
        if (pdl) {
            cudaLaunchAttribute &c = at[cfg->numAttrs++];
            c.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            c.val.programmaticStreamSerializationAllowed = 1;
        }
    }
};

// Host: the maps of a call's cache with boxes of `box` slots.
bool encode_cache(CacheMaps *maps, const Args &a, int type, int box);
// The queries as [token][head][d]: boxes of `tokens` tokens by a group's heads by 64 elements.
bool encode_queries(CUtensorMap *map, const Args &a, int type, int tokens);

}  // namespace attn
}  // namespace q4k
