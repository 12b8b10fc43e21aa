// 8-bit codes of a key/value cache as fp16 numbers, exactly.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "moe_q8k.h"

namespace moe {

// Two codes of a 32-bit word that lie in its bytes 1 and 3 (the other bytes do not matter), as an fp16 pair.
//   e4m3: s eeee mmm in the upper byte of each half, moved down by one bit below the sign: an fp16 number that is 2^-8
//         of the code's value (the biases are 15 and 7), subnormal codes included.  0x7f and 0xff are +-480.
//   int8: with the sign bit flipped, the byte v + 128 under the exponent of 1024 is 1152 + v.
// kCodeScale makes up for the first.
template <int FMT>
constexpr float kCodeScale = FMT == MOE_DT_E4M3 ? 256.0f : 1.0f;

__device__ __forceinline__ uint32_t half2_add(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int FMT>
__device__ __forceinline__ uint32_t upper_codes(uint32_t w) {
  if constexpr (FMT == MOE_DT_E4M3) return (w & 0x80008000u) | ((w >> 1) & 0x3f803f80u);
  else return half2_add(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u, 0xe480e480u);  // (1024 + 128 + v) - 1152
}
// Four codes of a word: lo = its bytes 0 and 2, hi = its bytes 1 and 3.
template <int FMT>
__device__ __forceinline__ void four_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == MOE_DT_E4M3) {
    lo = upper_codes<FMT>(w << 8);
    hi = upper_codes<FMT>(w);
  } else {
    lo = half2_add((w & 0x00ff00ffu) ^ 0x64806480u, 0xe480e480u);
    hi = upper_codes<FMT>(w);
  }
}
// the same as fp32 numbers, in the order of the bytes
template <int FMT>
__device__ __forceinline__ void four_values(uint32_t w, float* v) {
  uint32_t lo, hi;
  four_codes<FMT>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  v[0] = a.x * kCodeScale<FMT>, v[1] = b.x * kCodeScale<FMT>, v[2] = a.y * kCodeScale<FMT>, v[3] = b.y * kCodeScale<FMT>;
}

}  // namespace moe
