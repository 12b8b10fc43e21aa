// 8-bit codes of a key/value cache as fp16 numbers, exactly.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "moe_q8k.h"

namespace moe {

__device__ __forceinline__ uint32_t half2_add(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {  // of the two lower bytes
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(w));
  return r;
}

// Four codes of a word as two fp16 pairs.
//   e4m3: by the conversion instruction; lo = bytes 0 and 1, hi = bytes 2 and 3
//   int8: with the sign bit flipped, the byte v + 128 under the exponent of 1024 is 1152 + v;
//         lo = bytes 0 and 2, hi = bytes 1 and 3
template <int FMT>
__device__ __forceinline__ void four_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == MOE_DT_E4M3) {
    lo = e4m3_pair(w);
    hi = e4m3_pair(w >> 16);
  } else {
    lo = half2_add((w & 0x00ff00ffu) ^ 0x64806480u, 0xe480e480u);  // (1024 + 128 + v) - 1152
    hi = half2_add(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u, 0xe480e480u);
  }
}
// Bytes Z and Z + 1 of the words of two keys, each as the pair (first key, second key).
template <int FMT, int Z>
__device__ __forceinline__ void two_keys(uint32_t w0, uint32_t w1, uint32_t& first, uint32_t& second) {
  if constexpr (FMT == MOE_DT_E4M3) {
    const uint32_t x = __byte_perm(w0, w1, Z == 0 ? 0x5140 : 0x7362);
    first = e4m3_pair(x);
    second = e4m3_pair(x >> 16);
  } else {
    const uint32_t x = __byte_perm(w0, w1, Z == 0 ? 0x0400 : 0x0602), y = __byte_perm(w0, w1, Z == 0 ? 0x0501 : 0x0703);
    first = half2_add((x & 0x00ff00ffu) ^ 0x64806480u, 0xe480e480u);
    second = half2_add((y & 0x00ff00ffu) ^ 0x64806480u, 0xe480e480u);
  }
}
// The same where no result may be a NaN: e4m3's 0x7f and 0xff become +-480.  A byte s eeee mmm in the upper half of a
// 16-bit number, moved down by one bit below the sign, is 2^-8 of the code's value in fp16 (the biases are 15 and 7).
template <int FMT, int Z>
__device__ __forceinline__ void two_keys_finite(uint32_t w0, uint32_t w1, uint32_t& first, uint32_t& second) {
  if constexpr (FMT == MOE_DT_E4M3) {
    const uint32_t x = __byte_perm(w0, w1, Z == 0 ? 0x4404 : 0x6626), y = __byte_perm(w0, w1, Z == 0 ? 0x5515 : 0x7737);
    first = half2_mul((x & 0x80008000u) | ((x >> 1) & 0x3f803f80u), 0x5c005c00u);
    second = half2_mul((y & 0x80008000u) | ((y >> 1) & 0x3f803f80u), 0x5c005c00u);
  } else {
    two_keys<FMT, Z>(w0, w1, first, second);
  }
}
// four codes as fp32 numbers, in the order of the bytes
template <int FMT>
__device__ __forceinline__ void four_values(uint32_t w, float* v) {
  uint32_t lo, hi;
  four_codes<FMT>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  if constexpr (FMT == MOE_DT_E4M3) v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  else v[0] = a.x, v[1] = b.x, v[2] = a.y, v[3] = b.y;
}

}  // namespace moe
