// Microscaled 4-bit blocks (e2m1 codes under a power of two, include/moda.h) as bf16
// pairs, exactly.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "sm103.cuh"

namespace moda {
namespace mx4 {

// bf16 pairs: bit 15 or 31 set where a half is an infinity or a NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// 8 codes of a word times a power of two given as a bf16 pair (scale_of), as bf16 pairs in
// their order. Exact but at the ends of bf16's range, where it rounds to subnormals and
// infinities. (Conversions to fp16 and fp32 and back take half of the ALU's slots of what
// placing the code's bits takes: a 4-bit prefill's blocks 3700 cycles with that.)
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t scale, uint32_t (&out)[4]) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    out[i] = mul_bf16x2(sm103::pack_bf16x2(f.x, f.y), scale);
  }
}
// A block's scale byte b as a bf16 pair of 2^(b - 127); 255 is NaN.
__device__ __forceinline__ uint32_t scale_of(uint32_t b) {
  const uint32_t x = b == 255u ? 0x7fc0u : b == 0u ? 0x0040u : b << 7;
  return x | x << 16;
}
// The same in units of 2^unit; 0 where that is below 2^-126. (With the subnormals a 4-bit
// prefill of 1024 tokens at 32768 rows took 301 us, without 284.)
__device__ __forceinline__ uint32_t scale_in_units(uint32_t b, int unit) {
  const uint32_t x = b == 255u ? 0x7fc0u : (uint32_t)max((int)b - unit, 0) << 7;
  return x | x << 16;
}

}  // namespace mx4
}  // namespace moda
