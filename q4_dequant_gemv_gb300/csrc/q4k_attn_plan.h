// q4k_attn_plan.h -- which attention kernel, tile and way of joining a call takes.
//
// A call has tiles (some query rows of a sequence and cache head), each over
// units of keys.  Three ways to run them:
//   * few-rows kernel, a cluster of S CTAs per tile: waves of as many clusters as
//     fit at once, each start + join, and its rank's units;
//   * few-rows kernel, all units split evenly over the SMs: start, scratch and a
//     second launch to join, then a start per tile and the units;
//   * many-rows kernel (tcgen05), 256 rows a tile, split the same way.
// Small tiles fill the GPU and read keys again (from L2), large ones read them
// once.  The estimate below, in us, was fitted to 1317 measured calls (1 to 64
// sequences of 1 to 8 tokens, 28/4, 32/8 and 16/2 heads of 128, 16/16 of 64, 200 to
// 30000 positions, 16-bit and fp32 queries, page tables just wide enough), each in
// every form: for those calls its choice is within 1.2 % of the fastest on the
// geometric mean (1.4x at worst), where the rule before it (the smallest tile that
// holds a sequence's rows, clusters by units, the tcgen05 kernel above 16 rows) was
// 16 % off.  More than 8 tokens a sequence lie outside the fit.  Both sides, in us:
//   4 sequences of 5 x 7 rows over 2000: clusters with tiles of 8 rows 15, of 16 22, of 32 24;
//   64 of 8 x 7 over 200, fp32 queries: tiles of 8 70, of 16 51, of 32 44;
//   1 of 1 x 7 over 1000: cluster 7.2, split 12.3; 1 of 1 x 4 over 131072: 109 and 92;
//   2 x 4 rows over 14336, 16 bits: few-rows 20, many-rows 26; 8 x 4 rows 41 and 31.
// It knows no lengths, only what a page table row can hold.  A table much wider than
// the sequences makes it take them for long ones: one token of 28 / 4 heads over
// 1000 positions takes 7.1 us with a table of 1000, 11.2 (split, the cluster form
// still 7.1) with one of 16384 or more; sixteen over 4096 28.2 and, in a table of
// 32768, 36.1 (clusters 27.9).  Such a caller can ask for the form.
// 8-bit caches take the same estimate, with their widening added to the many-rows form
// (`widened_us`).  Over 216 bf16 calls of theirs (1 to 64 sequences of 2 to 128 tokens, 32/8
// and 28/4 heads of 128, 500 to 32000 positions, tables just wide enough, int8 in blocks of 16
// and e4m3 of 1) its choice is within 1.4 % of the fastest form on the geometric mean, 1.29x at
// worst (without that term 6.5 % and 2.1x); over 56 in tables eight times as wide 8 % and 1.9x
// (21 % and 2.1x).  Both sides, in us:
//   64 sequences of 4 tokens over 500, 28/4 heads: clusters of tiles of 32 rows 38, many-rows 82;
//   4 of 8 over 8000, 32/8: 50 and 80; 4 of 32 over 8000, 28/4: 146 and 59.
// (Their tiles of 8 rows have units of twice the keys that is counted here.)
#pragma once
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/q4k.h"
#include "q4k_attn_chunk.cuh"
#include "q4k_attn_rows.cuh"

namespace q4k {
namespace attn {

// Costs of a tile shape: us per unit (at one part, per further part), per wave of
// clusters, per tile of a split, per split call.
struct Cost {
    int rows;
    double unit, part, wave, tile, split;
};
constexpr Cost kCosts[] = {{8, 0.83, 0.11, 5.0, 3.0, 9.5}, {16, 1.05, 0.25, 5.7, 4.0, 11.3}, {32, 1.0, 0.23, 7.5, 5.0, 18.0}};
// A split: per further CTA of a tile (the join), where shares cut through tiles.
constexpr double kJoinPart = 0.2, kCut = 4.0;
constexpr double kChunkCall = 14.0, kChunkTile = 4.5, kChunkUnit = 1.35;

inline int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }

// form: Q4K_ATTN_* (0: any); room: clusters of 1 .. kMaxCluster CTAs that the GPU holds at once; parts: 16-bit parts of
// the queries.  A form that the call cannot take gives neither chunk nor rows.
inline Choice choose(const Args &a, const int (&room)[kMaxCluster + 1], int sms, int parts, bool may_chunk, int form = 0)
{
    Choice best{};
    double least = 1e300;
    // keys that a token can see, about: a window's (a prefix may reach past it)
    int64_t keys = a.capacity;
    if (a.window > 0) keys = std::min<int64_t>(keys, int64_t{a.window} + up(a.tokens, a.batch));
    const double small = a.dim <= 64 ? 0.7 : 1.0, small_split = a.dim <= 64 ? 1.1 : 1.0;
    auto join = [&](int64_t tiles, int64_t units) {
        const double ctas = std::min<double>(sms, 0.5 * static_cast<double>(tiles * units));
        return kJoinPart * std::max(0.0, ctas / static_cast<double>(tiles) - 1.0);
    };
    // tiles of a sequence of average length; where lengths differ some have one more
    const double slack = a.tokens % a.batch ? 1.15 : 1.0;
    const int64_t rows = static_cast<int64_t>(a.tokens) * a.group;
    for (int i = 0; i < 3; ++i) {
        const Cost &c = kCosts[i];
        const bool clusters = !form || form == Q4K_ATTN_CLUSTER8 + i, split = !form || form == Q4K_ATTN_SPLIT8 + i;
        if (a.dim > 128 && c.rows > 16) break;   // (registers)
        const int64_t unit = kBlock * (a.dim > 128 || c.rows > 16 ? 4 : 8), units = (keys + kBlock - 1) / unit + 1;
        const int64_t tiles = int64_t{a.kv_heads} * a.batch * up(rows, int64_t{c.rows} * a.batch);
        const double each = c.unit + c.part * (parts - 1);
        for (int S = 1; clusters && S <= kMaxCluster && S <= units; ++S) {
            // (a launch has a cluster for every tile that the lengths could make)
            if (room[S] < 1 || (rows / c.rows + a.batch) * a.kv_heads * S >= (1 << 24)) continue;
            const int64_t waves = up(static_cast<int64_t>(std::ceil(static_cast<double>(tiles) * slack)), room[S]);
            const double us = 2.0 + static_cast<double>(waves) * (c.wave + each * small * static_cast<double>(up(units, S)));
            if (us < least) least = us, best = {false, c.rows, S};
        }
        const double us = c.split + (tiles >= sms || sms % tiles ? kCut : 0.0) + join(tiles, units) +
                          static_cast<double>(tiles) / sms * (c.tile + each * small_split * static_cast<double>(units));
        if (split && us < least) least = us, best = {false, c.rows, 0};
    }
    if (may_chunk && (!form || form == Q4K_ATTN_MANY)) {
        const int64_t tiles = int64_t{a.kv_heads} * a.batch * up(a.tokens, int64_t{kChunkRows / a.group} * a.batch);
        const double us = kChunkCall + (a.ks ? widened_us(a, keys) : 0.0) + join(tiles, keys / kChunkKeys + 1) +
                          static_cast<double>(tiles) / sms * (a.dim <= 64 ? 0.8 : 1.0) *
                              (kChunkTile + kChunkUnit * static_cast<double>(keys / kChunkKeys + 1));
        if (us < least) best = {true, 0, 0};
    }
    return best;
}

}  // namespace attn
}  // namespace q4k
