// q4k_cache8.cuh -- the codes of an 8-bit cache (Q4K_I8, Q4K_E4M3) and their values.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/q4k.h"

namespace q4k {
namespace cache8 {

constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126: its reciprocal is finite

__device__ __forceinline__ float top_of(int codes) { return codes == Q4K_I8 ? 127.0f : 448.0f; }

// |x|, 0 for infinities and NaN.
__device__ __forceinline__ float finite_size(float x)
{
    const float s = fabsf(x);
    return s <= 3.402823466e38f ? s : 0.0f;
}

// Four codes of values that are already over their scale.
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], int codes)
{
    if (codes == Q4K_I8) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = x[j] == x[j] ? __float2int_rn(fminf(fmaxf(x[j], -127.0f), 127.0f)) : 0;
            w |= (static_cast<uint32_t>(c) & 0xFFu) << 8 * j;
        }
        return w;
    }
    uint16_t lo, hi;   // (the first operand is the upper half)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
    return static_cast<uint32_t>(hi) << 16 | lo;
}

// Two e4m3 codes as fp16 (exact).
__device__ __forceinline__ uint32_t e4m3_pair(uint16_t c)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return h;
}

__device__ __forceinline__ void decode4(uint32_t w, int codes, float (&f)[4])
{
    if (codes == Q4K_I8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = static_cast<float>(static_cast<int8_t>(w >> 8 * j & 0xFFu));
    } else {
        const uint32_t a = e4m3_pair(static_cast<uint16_t>(w)), b = e4m3_pair(static_cast<uint16_t>(w >> 16));
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a)), y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
        f[0] = x.x, f[1] = x.y, f[2] = y.x, f[3] = y.y;
    }
}

}  // namespace cache8
}  // namespace q4k
