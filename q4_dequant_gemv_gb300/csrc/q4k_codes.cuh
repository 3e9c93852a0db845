// q4k_codes.cuh -- codes of an 8-bit cache as operands of fp16 products.
#pragma once
#include <cstdint>

#include "../../include/q4k.h"
#include "ptx.cuh"
#include "q4k_cache8.cuh"

namespace q4k {
namespace attn {

// Codes of both a block's keys and its values as fp16 pairs.  Keys: four consecutive
// bytes of a row as two pairs.
template <int CT>
__device__ __forceinline__ void key_pairs(uint32_t w, uint32_t &p, uint32_t &q)
{
    if constexpr (CT == Q4K_I8) {   // 1024 + (code + 128) is 0x6400 | byte; minus 1152
        const uint32_t u = w ^ 0x80808080u;
        p = hsub2_u32(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
        q = hsub2_u32(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
    } else {
        p = cache8::e4m3_pair(static_cast<uint16_t>(w)), q = cache8::e4m3_pair(static_cast<uint16_t>(w >> 16));
    }
}

// Values: bytes 0, 1 (HIGH: 2, 3) of two rows, paired across the rows.
template <int CT, bool HIGH>
__device__ __forceinline__ void value_pairs(uint32_t w0, uint32_t w1, uint32_t &p, uint32_t &q)
{
    if constexpr (CT == Q4K_I8) {
        const uint32_t x = __byte_perm(w0, w1, HIGH ? 0x7632 : 0x5410);
        p = hsub2_u32((x & 0x00FF00FFu) ^ 0x64806480u, 0x64806480u);
        q = hsub2_u32((x >> 8 & 0x00FF00FFu) ^ 0x64806480u, 0x64806480u);
    } else {
        const uint32_t x = __byte_perm(w0, w1, HIGH ? 0x7362 : 0x5140);
        p = cache8::e4m3_pair(static_cast<uint16_t>(x)), q = cache8::e4m3_pair(static_cast<uint16_t>(x >> 16));
    }
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// 16 bytes global -> shared, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// 4 bytes global -> shared, or zeros.
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}

// A power of two from its exponent (-126 .. 127).
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

}  // namespace attn
}  // namespace q4k
