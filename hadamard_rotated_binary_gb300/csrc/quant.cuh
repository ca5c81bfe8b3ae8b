// The 4-bit form of a cache's heads (not part of the C-ABI).
//
// A head's D elements are four groups of D / 4 with a scale each.  A scale has
// 5 bits of exponent and 3 of significand: a float16 without its sign and last
// 7 bits, so byte << 7 is that float16.  A value is (nibble - 8) * scale with
// nibbles 1..15; its 3 + 4 significant bits are exact in bf16 and f16 alike, so
// every path reads the same values, whatever type it multiplies in.  Scales go
// up to 60: dequantisation is one fused multiply-add on the float16 1024 + nibble,
// whose constant -1032 * scale has to stay finite.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace bitlin_impl {

constexpr int kQuantGroups = 4;
constexpr uint32_t kQuantTopScale = 167;  // 60

__device__ __forceinline__ float quant_scale(uint32_t byte) { return __half2float(__ushort_as_half((unsigned short)(byte << 7))); }

// The scale nearest to amax / 7 (ties to even), decided on exact products: 7 times
// the middle of two scales has 8 significant bits.  T: float or double.
template <typename T>
__device__ __forceinline__ uint32_t quant_scale_code(T amax)
{
    const uint32_t low = __half_as_ushort(__float2half_rz((float)amax * (1.f / 7.f))) >> 7;
    if (low >= kQuantTopScale) return kQuantTopScale;
    const T middle = (T)7 * (T)(0.5f * (quant_scale(low) + quant_scale(low + 1)));
    return low + (amax > middle || (amax == middle && (low & 1)));
}

// Small integers to floats by joining them with a larger float's significand bits and taking that
// float away again is a published conversion (Kim, Henry, Fahim and Awadalla, "Who Says Elephants
// Can't Run", 2022, for 4 and 8 bits); the group's scale in its constants is this format's.
//
// Two nibbles of the same place in a word's halves, as f16 pairs: both of
// (word & 0x000f000f) through `low`, of (word & 0x00f000f0) through `high`.
struct QuantScale2 {
    __half2 low, low_add, high, high_add;
};
__device__ __forceinline__ QuantScale2 quant_scale2(uint32_t pair_of_bytes)  // one in each half
{
    const uint32_t bits = pair_of_bytes << 7;
    const __half2 s = *reinterpret_cast<const __half2*>(&bits);
    QuantScale2 q;
    q.low = s;
    q.low_add = __hmul2(s, __float2half2_rn(-1032.f));
    q.high = __hmul2(s, __float2half2_rn(0.0625f));
    q.high_add = __hmul2(s, __float2half2_rn(-72.f));
    return q;
}
// `magic` is 0x64006400, two float16 1024s, in a register: masked and joined in one
// operation (as a constant it would take a second one beside the mask).
__device__ __forceinline__ __half2 quant_low(uint32_t word, const QuantScale2& s, uint32_t magic)
{
    uint32_t bits;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(bits) : "r"(word), "r"(magic));
    return __hfma2(*reinterpret_cast<const __half2*>(&bits), s.low, s.low_add);
}
__device__ __forceinline__ __half2 quant_high(uint32_t word, const QuantScale2& s, uint32_t magic)
{
    uint32_t bits;
    asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(bits) : "r"(word), "r"(magic));
    return __hfma2(*reinterpret_cast<const __half2*>(&bits), s.high, s.high_add);
}

}  // namespace bitlin_impl
