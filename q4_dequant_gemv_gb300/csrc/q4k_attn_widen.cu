// q4k_attn_widen.cu -- prompt chunks over an 8-bit cache: the keys and values that the
// call may see go to fp16 once, then the many-rows kernel runs over them.
//
// That kernel's products want fp16 operands.  Turned inside it, each of a tile's 256 rows
// a code would cost as many instructions as its softmax does, again for every tile of a
// sequence (issue slots bound it at half the speed of a 16-bit cache: 2048 tokens over
// 14336 took 537 us at best); turned once they cost a read of the codes and a write and
// re-reads, mostly from L2, of twice as many bytes.
//
// Layout: pages of 128 positions, table_pages a sequence, [page][head][128][dim], and
// for each page and head the factors of its eight pieces of 16 keys, then of values.  A
// block of 16 tokens or more covers whole pieces: the factor is its scale, and the fp16
// values are the codes themselves, exactly.  Smaller blocks' scales multiply the codes over
// a power of two of the piece, its factor, with one rounding to fp16 (2^-11 of a value).  A piece
// that is not in the cache has factors of -inf; the kernel knows whether a row sees it.
// bf16 queries become fp16 over a power of two a row here too.
//
// What no token sees may hold any scale: it is not read where a window or (blocks below 16,
// whose scales share a power of two) kv_start leaves it out, else the attention kernel's
// factor warp lets it count as 0.
//
// 3 bytes a code and 4 an element of the queries.  Three chunks of 512 (1327 tokens) over up
// to 4608, 28 / 4 heads of 128 (12.4 M codes, 56 MB): 16 us of the call's 110 (the kernel 79,
// its join 22, each by itself), 3.5 TB/s: latency and issue slots (49 %), DRAM is at 17 %;
// 2048 over 14336, 32 / 8 heads (34 M codes, 134 MB) 27 of 395 (347, 20), 5 TB/s; with the
// conversion inside the kernel they took 142 and 537, the mma.sync kernel takes 753 for
// the first.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/q4k.h"
#include "q4k_attn_chunk.cuh"
#include "q4k_codes.cuh"

namespace q4k {
namespace attn {

constexpr int64_t kWidenLeast = int64_t{64} << 20;   // (a pass of no more than this many bytes is not divided)
constexpr int kWidenThreads = 256, kWidenWarps = kWidenThreads / 32, kPage = 128;
static_assert(kPage == kChunkKeys, "a unit of the many-rows kernel");

struct WidenArgs {
    Args a;                // of the call (k, v: codes; heads of this pass)
    __half *k, *v, *q;     // to (q: null if the queries are fp16)
    float *factors, *row_scale;
};

// Sixteen codes as fp16, times s (0: as they are).
template <int CODES>
__device__ __forceinline__ void widen16(const uint4 &raw, float s, uint4 &x, uint4 &y)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        key_pairs<CODES>(w[i], r[2 * i], r[2 * i + 1]);
        if (s != 0.0f) {
#pragma unroll
            for (int j = 2 * i; j < 2 * i + 2; ++j) {   // (fp32 product, one rounding)
                const float2 f = unpack2(r[j], Q4K_F16);
                r[j] = pack2(f.x * s, f.y * s, Q4K_F16);
            }
        }
    }
    x = make_uint4(r[0], r[1], r[2], r[3]), y = make_uint4(r[4], r[5], r[6], r[7]);
}

// A piece of 16 positions, head and side: a warp.  `live`: the piece's rows that count.
__device__ __forceinline__ void widen_piece(const WidenArgs &w, int64_t to, int piece, int head, int side, int page, int slot, uint32_t live)
{
    const Args &a = w.a;
    const int lane = threadIdx.x & 31;
    const float *scales = side ? a.vs + page * a.vs_page + head * a.vs_head : a.ks + page * a.ks_page + head * a.ks_head;
    const int64_t block = side ? a.vs_block : a.ks_block, slots = side ? a.v_slot : a.k_slot;
    // the codes first: rows of CPR chunks (plain loads: as a programmatic dependent this kernel starts while the append
    // before it still writes them)
    const int cpr = a.dim > 64 ? 8 : 4, rps = 32 / cpr, ch = lane & (cpr - 1), row0 = lane / cpr;
    const uint8_t *from = static_cast<const uint8_t *>(side ? a.v : a.k) + page * (side ? a.v_page : a.k_page) +
                          head * (side ? a.v_head : a.k_head) + (slot + row0) * slots + 16 * ch;
    const bool inside = 16 * ch < a.dim;
    uint4 raw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (inside && rps * j < 16 && (live >> (row0 + rps * j) & 1)) raw[j] = *reinterpret_cast<const uint4 *>(from + j * rps * slots);
    }
    float s = 0.0f, factor;   // s: of row lane % 16, over the factor; 0 where the codes stay
    if (a.block_shift >= 4) {
        factor = scales[(slot >> a.block_shift) * block];
        if (factor < 0.0f) s = -1.0f, factor = -factor;   // (factors have no sign: the codes take it)
    } else {
        const int r = lane & 15;
        s = live >> r & 1 ? scales[((slot + r) >> a.block_shift) * block] : 0.0f;
        float most = fabsf(s);
#pragma unroll
        for (int o = 8; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const int x = max(-120, min(115, static_cast<int>(__float_as_uint(most) >> 23) - 133));   // the largest to [64, 128)
        s *= two_to(-x);
        factor = most > 0.0f ? two_to(x) : 0.0f;
    }
    if (lane == 0) w.factors[to * 16 + 8 * side + piece] = factor;
    __half *out = (side ? w.v : w.k) + (to * kPage + 16 * piece) * a.dim + 16 * ch;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = row0 + rps * j;
        const float f = __shfl_sync(0xffffffffu, s, r & 15);
        if (!inside || rps * j >= 16 || !(live >> r & 1)) continue;
        uint4 x, y;
        if (a.codes == Q4K_I8) widen16<Q4K_I8>(raw[j], f, x, y);
        else widen16<Q4K_E4M3>(raw[j], f, x, y);
        // (a row of scale 0 among scaled ones: its codes count for nothing)
        if (a.block_shift < 4 && f == 0.0f) x = y = make_uint4(0, 0, 0, 0);
        uint4 *p = reinterpret_cast<uint4 *>(out + static_cast<int64_t>(r) * a.dim);
        p[0] = x, p[1] = y;
    }
}

// blockIdx.y = the sequence, its pieces in strides of the grid; one more: the queries.
__global__ void __launch_bounds__(kWidenThreads) widen_kernel(const __grid_constant__ WidenArgs w)
{
    const Args &a = w.a;
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
    if (b == a.batch) {
        // rows of dim / 8 lanes in groups of 16 (8)
        const int lanes = a.dim > 64 ? 16 : 8, per = 32 / lanes, c = lane & (lanes - 1);
        const int64_t rows = static_cast<int64_t>(a.tokens) * a.heads;
        for (int64_t r = (static_cast<int64_t>(blockIdx.x) * kWidenWarps + warp) * per; r < rows;
             r += static_cast<int64_t>(gridDim.x) * kWidenWarps * per) {
            const int64_t row = r + lane / lanes, tok = row / a.heads, h = row - tok * a.heads;
            uint4 raw = make_uint4(0, 0, 0, 0);
            const bool here = row < rows && 8 * c < a.dim;
            if (here) raw = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + tok * a.q_token + h * a.q_head + 8 * c);
            const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
            float mx = 0.0f;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const float2 f = unpack2(u[z], a.q_type);
                mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            for (int o = lanes >> 1; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const int ex = static_cast<int>(__float_as_uint(mx) >> 23);
            const int e = ex != 0 && ex != 255 ? max(-126, min(126, 141 - ex)) : 0;   // max|q| to [2^14, 2^15)
            const float up = two_to(e);
            if (here) {
                uint32_t v[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const float2 f = unpack2(u[z], a.q_type);
                    v[z] = pack2(f.x * up, f.y * up, Q4K_F16);
                }
                *reinterpret_cast<uint4 *>(w.q + row * a.dim + 8 * c) = make_uint4(v[0], v[1], v[2], v[3]);
                if (c == 0) w.row_scale[row] = two_to(-e);
            }
        }
        return;
    }
    // what the sequence's tokens may see: from its first token's window on
    auto start_of = [&](int i) { return min(max(a.seq_start[i], 0), a.tokens); };
    const int s0 = start_of(b), n = start_of(b + 1) - s0, raw_len = a.kv_len[b];
    if (n <= 0) return;
    const int len = min(max(raw_len, 0), a.capacity), first = max(raw_len, -1) - n;
    int lo = a.window ? min(max(first + 1 - a.window, 0), len) : 0;
    // Blocks below 16: the scales of a piece meet over one power of two, so those that no token sees, which may be
    // anything, have to stay out.  What is seen has no holes unless a token does not see its own position.
    const bool starts = a.kv_start && a.block_shift < 4;
    bool holes = false;
    if (starts) {
        __shared__ int s_lo, s_holes;
        if (threadIdx.x == 0) s_lo = len, s_holes = 0;
        __syncthreads();
        int least = len;
        for (int i = threadIdx.x; i < n; i += kWidenThreads) {
            const Range r = token_range(a, b, first + i, s0 + i, len);
            if (r.hi > r.lo) least = min(least, r.lo);
            holes |= a.causal && r.lo > first + i;
        }
        atomicMin(&s_lo, least);
        if (holes) s_holes = 1;
        __syncthreads();
        lo = s_lo, holes = s_holes != 0;
    }
    auto seen16 = [&](int key) {   // which of 16 keys some token sees, whole warps
        uint32_t seen = 0;
        for (int i = lane; i < n; i += 32) {
            const Range r = token_range(a, b, first + i, s0 + i, len);
            seen |= span(r.lo - key, r.hi - key);
        }
        return __reduce_or_sync(0xffffffffu, seen);
    };
    // a warp per piece, head and side, neighbouring warps on neighbouring heads
    const int pg0 = lo / kPage, per_page = 16 * a.kv_heads;
    const int64_t tasks = len > pg0 * kPage ? static_cast<int64_t>((len + kPage - 1) / kPage - pg0) * per_page : 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWidenWarps + warp; i < tasks; i += static_cast<int64_t>(gridDim.x) * kWidenWarps) {
        const uint32_t x = static_cast<uint32_t>(quotient(i, a.kv_heads));   // (a position's fits 32 bits)
        const int head = static_cast<int>(i - static_cast<int64_t>(x) * a.kv_heads), side = x & 1, piece = x >> 1 & 7, pg = pg0 + (x >> 4);
        const int key = pg * kPage + 16 * piece;
        uint32_t live = span(lo - key, len - key) & 0xFFFFu;
        if (holes && live) live &= seen16(key);
        int page = -1, slot = 0;
        if (live) {
            int e;
            page_of(a, key, e, slot);
            page = a.page_table[b * a.table_stride + e];
        }
        const int64_t to = (static_cast<int64_t>(b) * a.table_pages + pg) * a.kv_heads + head;
        if (page >= 0 && page < a.pages) widen_piece(w, to, piece, head, side, page, slot, live);
        else if (lane == 0) w.factors[to * 16 + 8 * side + piece] = live ? -INFINITY : 0.0f;
    }
}

// Bytes of the widened keys, values and factors of one cache head of one sequence.
int64_t widened_bytes(const Args &a)
{
    return (a.capacity + static_cast<int64_t>(kPage) - 1) / kPage * (2 * kPage * 2 * static_cast<int64_t>(a.dim) + 64);
}

// Cache heads and sequences of a pass that holds `fit` heads of one sequence: heads of all sequences, or one head of
// as many as fit.  Passes of about the same size.
struct Pass {
    int heads, seqs;
};
static Pass pass_of(const Args &a, int64_t fit)
{
    auto alike = [](int n, int64_t most) {
        const int passes = static_cast<int>((n + most - 1) / most);
        return (n + passes - 1) / passes;
    };
    return {alike(a.kv_heads, std::max<int64_t>(1, fit / a.batch)), alike(a.batch, std::min<int64_t>({fit, a.batch, 65534}))};   // (a grid's y)
}

static int64_t fitting(const Args &a) { return std::max<int64_t>(1, kWidenMost / widened_bytes(a)); }

// What widening adds to a call that sees `keys` positions a sequence, about, in us: a launch, bytes (three a code, four an
// element of queries that are turned) and the start and end of each further pass.  Fitted with the estimate of the forms.
double widened_us(const Args &a, int64_t keys)
{
    const double codes = 2.0 * static_cast<double>(keys) * a.batch * a.kv_heads * a.dim;
    const double q = a.q_type == Q4K_F16 ? 0.0 : static_cast<double>(a.tokens) * a.heads * a.dim;
    const Pass p = pass_of(a, fitting(a));
    const double passes = static_cast<double>((a.kv_heads + p.heads - 1) / p.heads) * ((a.batch + p.seqs - 1) / p.seqs);
    return 6.0 + (3.0 * codes + 4.0 * q) / 7e6 + 45.0 * (passes - 1.0);
}

// In passes of what kWidenMost bytes hold; of less where the device has no room for that.
cudaError_t launch_widened(const ChunkLaunch &l)
{
    const Args &all = l.args;
    const int table_pages = (all.capacity + kPage - 1) / kPage;
    const bool turn = all.q_type != Q4K_F16;
    auto room = [](int64_t n) { return (n + 255) / 256 * 256; };
    int heads, seqs;
    int64_t pages, side, fac, q, scale;
    void *scratch = nullptr;
    cudaError_t e;
    for (int64_t fit = fitting(all);;) {
        const Pass p = pass_of(all, fit);
        heads = p.heads, seqs = p.seqs;
        pages = static_cast<int64_t>(seqs) * table_pages;
        side = room(pages * heads * kPage * all.dim * 2), fac = room(pages * heads * 64);
        const int64_t rows = static_cast<int64_t>(all.tokens) * heads * all.group;
        q = turn ? room(rows * all.dim * 2) : 0, scale = turn ? room(rows * 4) : 0;
        e = take_scratch(l.device, &scratch, 2 * side + fac + q + scale, l.stream, true);
        if (e != cudaErrorMemoryAllocation || 2 * side <= kWidenLeast || static_cast<int64_t>(heads) * seqs == 1) break;
        (void)cudaGetLastError();
        fit = std::max<int64_t>(1, static_cast<int64_t>(heads) * seqs / 2);
    }
    if (e != cudaSuccess) return e;
    uint8_t *at = static_cast<uint8_t *>(scratch);
    auto pass = [&](int h0, int b0) {
        WidenArgs w{};
        Args &a = w.a;
        a = all;
        a.kv_heads = std::min(heads, all.kv_heads - h0), a.heads = a.kv_heads * all.group, a.table_pages = table_pages;
        a.batch = std::min(seqs, all.batch - b0);
        a.seq_start += b0, a.kv_len += b0, a.page_table += b0 * all.table_stride;
        if (all.prefix_len) a.prefix_len += b0;
        a.k = static_cast<const uint8_t *>(all.k) + h0 * all.k_head, a.v = static_cast<const uint8_t *>(all.v) + h0 * all.v_head;
        a.ks += h0 * all.ks_head, a.vs += h0 * all.vs_head;
        const int64_t hq = static_cast<int64_t>(h0) * all.group;
        a.q = static_cast<const uint16_t *>(all.q) + hq * all.q_head, a.out = static_cast<uint16_t *>(all.out) + hq * all.out_head;
        if (all.lse) a.lse += hq;
        if (all.slopes) a.slopes += hq;
        w.k = reinterpret_cast<__half *>(at), w.v = reinterpret_cast<__half *>(at + side);
        w.factors = reinterpret_cast<float *>(at + 2 * side);
        if (turn) w.q = reinterpret_cast<__half *>(at + 2 * side + fac), w.row_scale = reinterpret_cast<float *>(at + 2 * side + fac + q);
        cudaLaunchConfig_t cfg = {};
        // up to eight CTAs an SM in all, each sequence's pieces dealt out over its share; the heads' queries once
        const bool queries = turn && b0 == 0;
        const int64_t q_ctas = queries ? (static_cast<int64_t>(all.tokens) * a.heads + 15) / 16 : 1;
        const int x = static_cast<int>(std::max<int64_t>(std::min<int64_t>(2 * static_cast<int64_t>(table_pages) * a.kv_heads,
                                                                           (8 * l.sms + a.batch - 1) / a.batch),
                                                         std::min<int64_t>(q_ctas, 4 * l.sms)));
        cfg.gridDim = dim3(static_cast<unsigned>(x), static_cast<unsigned>(a.batch + (queries ? 1 : 0)));
        cfg.blockDim = kWidenThreads;
        cfg.stream = l.stream;
        // (a later pass writes what the one before it reads)
        const Attributes attributes(&cfg, 0, all.pdl && h0 == 0 && b0 == 0);
        const cudaError_t err = cudaLaunchKernelEx(&cfg, widen_kernel, w);
        if (err != cudaSuccess) return err;
        ChunkLaunch ch = l;
        Args &c = ch.args;
        c = a;
        c.k = w.k, c.v = w.v, c.factors = w.factors, c.row_scale = w.row_scale;
        c.k_head = c.v_head = static_cast<int64_t>(kPage) * a.dim, c.k_slot = c.v_slot = a.dim;
        c.k_page = c.v_page = a.kv_heads * c.k_head;
        c.pages = static_cast<int>(pages), c.page_size = kPage, c.page_shift = 7;
        c.q_type = Q4K_F16, c.pdl = true;
        if (turn) c.q = w.q, c.q_head = a.dim, c.q_token = static_cast<int64_t>(a.heads) * a.dim;
        return launch_chunk_wide(ch);
    };
    for (int h0 = 0; h0 < all.kv_heads && e == cudaSuccess; h0 += heads)
        for (int b0 = 0; b0 < all.batch && e == cudaSuccess; b0 += seqs) e = pass(h0, b0);
    const cudaError_t f = cudaFreeAsync(scratch, l.stream);
    return e == cudaSuccess ? f : e;
}

}  // namespace attn
}  // namespace q4k
