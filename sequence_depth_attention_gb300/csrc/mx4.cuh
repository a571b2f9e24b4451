// Microscaled 4-bit blocks (e2m1 codes under a power of two, include/moda.h) as bf16
// pairs, exactly.
#pragma once

#include <stdint.h>

namespace moda {
namespace mx4 {

// bf16 pairs: bit 15 or 31 set where a half is an infinity or a NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// 8 codes of a word times 2^(byte - 127), as bf16 pairs. A code's three magnitude
// bits in bits 6 to 8 of a bf16 are its value times 2^-126 (a subnormal for 0.5),
// so one exact product by 2^(byte - 1) gives the value; above 2^127 the product is
// made in two steps.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t mul, uint32_t mul2, uint32_t (&out)[4]) {
  // halves hold codes j and j + 4
  uint32_t x[4];
  x[0] = ((w << 6) & 0x01c001c0u) | ((w << 12) & 0x80008000u);
  x[1] = ((w << 2) & 0x01c001c0u) | ((w << 8) & 0x80008000u);
  x[2] = ((w >> 2) & 0x01c001c0u) | ((w << 4) & 0x80008000u);
  x[3] = ((w >> 6) & 0x01c001c0u) | (w & 0x80008000u);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = mul_bf16x2(x[j], mul);
  if (mul2 != 0x3f803f80u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = mul_bf16x2(x[j], mul2);
  }
  out[0] = __byte_perm(x[0], x[1], 0x5410);
  out[1] = __byte_perm(x[2], x[3], 0x5410);
  out[2] = __byte_perm(x[0], x[1], 0x7632);
  out[3] = __byte_perm(x[2], x[3], 0x7632);
}
// The two factors for a scale byte, each in both halves: 2^(b - 1) up to b = 128,
// then 2^127 and 2^(b - 128); 255 is NaN.
__device__ __forceinline__ void factors(uint32_t b, uint32_t& mul, uint32_t& mul2) {
  const uint32_t e = min(b + 126u, 254u);  // biased exponent of the first; b = 0: 2^-1
  uint32_t m = e << 7, n = 0x3f80u;
  if (b > 128u) n = (b - 1u) << 7;         // 2^(b - 128)
  if (b == 255u) m = 0x7fc0u;
  mul = m | m << 16;
  mul2 = n | n << 16;
}

}  // namespace mx4
}  // namespace moda
