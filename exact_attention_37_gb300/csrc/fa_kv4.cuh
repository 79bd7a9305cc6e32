// From 4-bit codes to the values they stand for, two at a time.
#pragma once
#include <cstdint>

namespace fa {

// (a & mask) | magic
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(magic));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t fma16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  if constexpr (BF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Values of the four nibble pairs (k, k + 4) of x, k = 0..3: v[k] = (nibble k, nibble k + 4),
// with a scale and a low value for each half.
template <bool BF16>
__device__ __forceinline__ void values4(uint32_t x, uint32_t s2, uint32_t l2, uint32_t (&v)[4]) {
  if constexpr (BF16) {
    constexpr uint32_t kMagic = 0x43004300u, kOne = 0x3F803F80u, kMinus = 0xC300C300u;  // 128, 1, -128
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = fma16<true>(fma16<true>(and_or(x >> (4 * k), 0x000F000Fu, kMagic), kOne, kMinus), s2, l2);
  } else {
    constexpr uint32_t kMagic = 0x64006400u, kOne = 0x3C003C00u, kMinus = 0xE400E400u;  // 1024, 1, -1024
    constexpr uint32_t kSixteenth = 0x2C002C00u, kMinus64 = 0xD400D400u;                // 1/16, -64
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const uint32_t y = x >> (4 * k);
      v[k] = fma16<false>(fma16<false>(and_or(y, 0x000F000Fu, kMagic), kOne, kMinus), s2, l2);
      v[k + 1] = fma16<false>(fma16<false>(and_or(y, 0x00F000F0u, kMagic), kSixteenth, kMinus64), s2, l2);
    }
  }
}

// The same values times 2^-32, for bf16.  Four bits c at the bottom of a bf16 are the
// number c 2^-133, and four bits higher c 2^-129 (the step from subnormal to normal numbers
// is part of the line), so the codes need no exponent put above them and taken off again:
// with scale 2^101 and scale 2^97 one fused multiply-add gives 2^-32 (low + scale code),
// rounded once: 9 instructions for 8 values against 15.  2^-32 changes no bit of the
// mantissa of a value from 2^-94 on (one below is off by at most 2^-101), and the scales
// stay finite below 2^27.
constexpr float kScaledBack = 4294967296.f;
struct Scaled {
  uint32_t s0, s1, low;
  __device__ __forceinline__ static uint32_t mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ Scaled(uint32_t s2, uint32_t l2)
      : s0(mul(s2, 0x72007200u)), s1(mul(s2, 0x70007000u)), low(mul(l2, 0x2F802F80u)) {}  // 2^101, 2^97, 2^-32
};
__device__ __forceinline__ void values4_scaled(uint32_t x, const Scaled& p, uint32_t (&v)[4]) {
  v[0] = fma16<true>(x & 0x000F000Fu, p.s0, p.low);
  v[1] = fma16<true>(x & 0x00F000F0u, p.s1, p.low);
  v[2] = fma16<true>((x >> 8) & 0x000F000Fu, p.s0, p.low);
  v[3] = fma16<true>((x >> 8) & 0x00F000F0u, p.s1, p.low);
}

}  // namespace fa
