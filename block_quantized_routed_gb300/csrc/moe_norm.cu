// Residual addition, root-mean-square norm and an 8-bit output in one pass.
//
//   s = x + residual,  z = s * rsqrt(mean(s^2) + eps) * (w + offset)
//   q = codes of z with one scale per 256 / 128 columns or per row
//
// What bounds it: memory.  Every element of x and residual is read once and
// every output written once; s stays in registers between the sum of squares
// and the scaling, so there is no second pass over global memory.  8192 rows of
// 4096 (bf16 in, residual and sum; fp8 codes by 128 columns): 37 us, 6.4 TB/s.
// A few rows are latency: 37 of 6144 with codes by row 2.9 us.
//
// Layout: one CTA per row.  A thread holds NV vectors of 8 consecutive
// columns (vector i * blockDim + tid), so a warp's vectors are 256
// consecutive columns: a q8_K block is one warp-wide maximum, a group of 128
// columns a half-warp's, and neither needs shared memory.  Rows that are not
// 16-byte aligned (odd H, odd strides; WIDE = false) keep a warp's 256 columns,
// but a thread's eight are 32 apart, so that a warp's elements lie together
// (1715 rows of 7067, fp32 in, residual and sum: 29 us, 5.8 TB/s; 83 with eight
// consecutive ones).
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }

// A thread's 8 elements as fp32.  WIDE: consecutive, 16-byte aligned, all there.  Else 32 apart, as far as the row's
// `n` remaining columns go.
template <typename T, bool WIDE>
__device__ __forceinline__ void load8(const T* p, int n, float* v) {
  if constexpr (WIDE) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      T e[8];
      *reinterpret_cast<uint4*>(e) = a;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_f<T>(e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 32 * i < n ? to_f<T>(p[32 * i]) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T, bool WIDE>
__device__ __forceinline__ void store8(T* p, int n, const float* v) {
  if constexpr (WIDE) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(p) =
          make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * i < n) p[32 * i] = from_f<T>(v[i]);
  }
}

// the same with the type known at run time (uniform over the grid)
template <bool WIDE>
__device__ __forceinline__ void load8_dt(const void* p, int dt, int64_t at, int n, float* v) {
  if (dt == MOE_DT_F32) load8<float, WIDE>(static_cast<const float*>(p) + at, n, v);
  else if (dt == MOE_DT_BF16) load8<__nv_bfloat16, WIDE>(static_cast<const __nv_bfloat16*>(p) + at, n, v);
  else load8<__half, WIDE>(static_cast<const __half*>(p) + at, n, v);
}
template <bool WIDE>
__device__ __forceinline__ void store8_dt(void* p, int dt, int64_t at, int n, const float* v) {
  if (dt == MOE_DT_F32) store8<float, WIDE>(static_cast<float*>(p) + at, n, v);
  else if (dt == MOE_DT_BF16) store8<__nv_bfloat16, WIDE>(static_cast<__nv_bfloat16*>(p) + at, n, v);
  else store8<__half, WIDE>(static_cast<__half*>(p) + at, n, v);
}

// over a warp, in a fixed order: the sum of `sum` (SUM), the maximum of `peak` (MAX)
template <bool SUM, bool MAX>
__device__ __forceinline__ void warp_reduce(float& sum, float& peak) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if constexpr (SUM) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (MAX) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
  }
}
// the same over the block, for all its threads, behind one barrier
template <bool SUM, bool MAX>
__device__ __forceinline__ void block_reduce(float& sum, float& peak, float (&buf)[2][32]) {
  warp_reduce<SUM, MAX>(sum, peak);
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (nw == 1) return;
  if (lane == 0) {
    if constexpr (SUM) buf[0][threadIdx.x >> 5] = sum;
    if constexpr (MAX) buf[1][threadIdx.x >> 5] = peak;
  }
  __syncthreads();
  if constexpr (SUM) sum = lane < nw ? buf[0][lane] : 0.0f;
  if constexpr (MAX) peak = lane < nw ? buf[1][lane] : 0.0f;
  warp_reduce<SUM, MAX>(sum, peak);
}

// The q8_K rounding of z / d: half away from zero, clamped.  The product x
// with the reciprocal (1 ulp) is within 2 ulp of the IEEE quotient, which is at
// most 127: 2^-15.  Both round alike unless they are that near a half, and away
// from a half adding 1.5 * 2^23 rounds to the nearest, the code in the low byte.
// Near a half, or beyond the range, it is divided and rounded as written.
// Returns the bits of code + 1.5 * 2^23.
constexpr float kMagic = 12582912.0f;
__device__ __forceinline__ int q8k_bits(float z, float d, float inv) {
  const float x = z * inv;
  float y = x + kMagic;
  if (!(fabsf(x - (y - kMagic)) < 0.49996f)) y = fminf(127.0f, fmaxf(-127.0f, roundf(__fdiv_rn(z, d)))) + kMagic;
  return __float_as_int(y);
}

__device__ __forceinline__ float rcp(float x) {  // the approximation (1 ulp) and one Newton step: little over half an ulp
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return fmaf(y, fmaf(-x, y, 1.0f), y);
}

// the first column of a thread's vector i; the other seven follow it, or lie 32 apart
template <bool WIDE>
__device__ __forceinline__ int first_column(int i) {
  const int at = i * blockDim.x + threadIdx.x;
  return WIDE ? at * 8 : (at & ~31) * 8 + (at & 31);
}

// The 8-bit output of one row z = v * r (v in s[NV][8]; r = 1 but for fp8
// codes, which r does not change: they are v over the largest |v|, a rounding
// less).  `peak` is the row's largest |v| (row-scaled outputs only).  FMT: the
// format.  The scale d is an IEEE quotient; v / d is the
// product with d's reciprocal, which for int8 codes is put right near a half.
template <int NV, int FMT>
__device__ __forceinline__ void put_codes(const NormArgs& a, int64_t row, float (&s)[NV][8], float peak, float r) {
  const int tid = threadIdx.x, nt = blockDim.x;
  constexpr int fmt = FMT;
  constexpr bool fp8 = fmt == MOE_NORM_Q_E4M3_G128 || fmt == MOE_NORM_Q_E4M3_ROW;
  constexpr bool per_row = fmt == MOE_NORM_Q_E4M3_ROW || fmt == MOE_NORM_Q_INT8_ROW;
  const float top = fp8 ? 448.0f : 127.0f;
  float d = 0.0f;
  if (per_row) {
    d = __fdiv_rn(peak, top);
    if (tid == 0) a.d[row] = fp8 ? d * r : d;
  }
  const int group = fmt == MOE_NORM_Q_Q8K ? 256 : 128;
  uint8_t* const out = static_cast<uint8_t*>(a.q) + row * a.H;
  float* const dout = a.d + row * ((a.H + group - 1) / group);
  float m[NV];
  if (!per_row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      m[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m[i] = fmaxf(m[i], fabsf(s[i][j]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
    if (group == 256) {
#pragma unroll
      for (int i = 0; i < NV; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + tid) * 8, n = a.H - c;
    if (!per_row) {
      d = __fdiv_rn(m[i], top);
      if (n > 0 && c % group == 0) dout[c / group] = fp8 ? d * r : d;
    }
    // d = 0 only where every v of the group is 0 (or too small for its quotient to exist).  A reciprocal beyond
    // fp32 (d below 2^-126) is not used: such groups are divided.
    float inv = d > 0.0f ? rcp(d) : 0.0f, dq = d;
    if (d < 1.2e-38f && d > 0.0f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = __fdiv_rn(s[i][j], d);
      inv = dq = 1.0f;
    }
    uint32_t lo, hi;
    int sum = 0;
    if (fp8) {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        h[j / 2] = __nv_cvt_float2_to_fp8x2(make_float2(s[i][j] * inv, s[i][j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      lo = h[0] | h[1] << 16;
      hi = h[2] | h[3] << 16;
    } else {
      int code[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        code[j] = q8k_bits(s[i][j], dq, inv);
        sum += code[j];
      }
      sum -= 8 * __float_as_int(kMagic);
      lo = __byte_perm(__byte_perm(code[0], code[1], 0x0040), __byte_perm(code[2], code[3], 0x0040), 0x5410);
      hi = __byte_perm(__byte_perm(code[4], code[5], 0x0040), __byte_perm(code[6], code[7], 0x0040), 0x5410);
    }
    if (n > 0) *reinterpret_cast<uint2*>(out + c) = make_uint2(lo, hi);
    if (fmt == MOE_NORM_Q_Q8K && a.bsum16) {  // two lanes hold the 16 codes
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      if (n > 0 && (tid & 1) == 0) a.bsum16[row * (a.H / 16) + c / 16] = (int16_t)sum;
    }
  }
}

// The same for rows off the 16-byte boundaries: a thread's elements are 32
// columns apart, so a vector's first four lie in one group of 128, the others
// in the next.
template <int NV>
__device__ __forceinline__ void put_codes_narrow(const NormArgs& a, int64_t row, const float (&s)[NV][8], float peak,
                                                 float r) {
  const int lane = threadIdx.x & 31, fmt = a.q_fmt;
  const bool fp8 = fmt == MOE_NORM_Q_E4M3_G128 || fmt == MOE_NORM_Q_E4M3_ROW;
  const bool per_row = fmt == MOE_NORM_Q_E4M3_ROW || fmt == MOE_NORM_Q_INT8_ROW;
  const float top = fp8 ? 448.0f : 127.0f;
  const int group = fmt == MOE_NORM_Q_Q8K ? 256 : 128;
  uint8_t* const out = static_cast<uint8_t*>(a.q) + row * a.H;
  float* const dout = a.d + row * ((a.H + group - 1) / group);
  float d[2] = {0.0f, 0.0f};
  if (per_row) {
    d[0] = d[1] = __fdiv_rn(peak, top);
    if (threadIdx.x == 0) a.d[row] = fp8 ? d[0] * r : d[0];
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first_column<false>(i), n = a.H - c;
    if (!per_row) {
      float m[2] = {0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j / 4] = fmaxf(m[j / 4], fabsf(s[i][j]));
      if (group == 256) m[0] = m[1] = fmaxf(m[0], m[1]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int h = 0; h < 2; ++h) m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], o));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        d[h] = __fdiv_rn(m[h], top);
        if (lane == 0 && 128 * h < n && 128 * h % group == 0) dout[(c + 128 * h) / group] = fp8 ? d[h] * r : d[h];
      }
    }
    float inv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) inv[h] = d[h] > 0.0f ? rcp(d[h]) : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = s[i][j], dq = d[j / 4], x = inv[j / 4];
      if (dq < 1.2e-38f && dq > 0.0f) v = __fdiv_rn(v, dq), dq = x = 1.0f;  // as above
      int code;
      if (fp8) code = __nv_cvt_float_to_fp8(v * x, __NV_SATFINITE, __NV_E4M3);
      else code = q8k_bits(v, dq, x) - __float_as_int(kMagic);
      if (32 * j < n) out[c + 32 * j] = (uint8_t)code;
      if (fmt == MOE_NORM_Q_Q8K && a.bsum16) {  // 16 lanes hold the 16 codes
        int sum = code;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if ((lane & 15) == 0 && 32 * j < n) a.bsum16[row * (a.H / 16) + (c + 32 * j) / 16] = (int16_t)sum;
      }
    }
  }
}

// two fp32 operations in one instruction (each rounded as the scalar one)
__device__ __forceinline__ uint64_t bits2(float2 v) {
  return (uint64_t)__float_as_uint(v.x) | (uint64_t)__float_as_uint(v.y) << 32;
}
__device__ __forceinline__ float2 unbits2(uint64_t v) {
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return unbits2(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return unbits2(d);
}
__device__ __forceinline__ void add2(float* a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(make_float2(a[0], a[1]))), "l"(bits2(b)));
  const float2 r = unbits2(d);
  a[0] = r.x;
  a[1] = r.y;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4* v, float* f) {
  if constexpr (sizeof(T) == 4) {
    const uint4 x = v[0], y = v[1];
    f[0] = __uint_as_float(x.x), f[1] = __uint_as_float(x.y), f[2] = __uint_as_float(x.z), f[3] = __uint_as_float(x.w);
    f[4] = __uint_as_float(y.x), f[5] = __uint_as_float(y.y), f[6] = __uint_as_float(y.z), f[7] = __uint_as_float(y.w);
  } else {
    const uint4 x = v[0];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = t.x, f[2 * i + 1] = t.y;
      }
    }
  }
}
// FMT: the 8-bit format, or -1 for a.q_fmt (rows that are not WIDE)
template <typename XT, typename RT, int NV, bool WIDE, int FMT>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512, NV == 2 ? 2 : 1) add_rmsnorm_kernel(const NormArgs a) {
  __shared__ float buf[2][32];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int fmt = FMT >= 0 ? FMT : a.q_fmt;
  const bool per_row = fmt == MOE_NORM_Q_E4M3_ROW || fmt == MOE_NORM_Q_INT8_ROW;
  const XT* x = static_cast<const XT*>(a.x) + row * a.x_stride;
  const RT* res = static_cast<const RT*>(a.residual) + row * a.r_stride;
  RT* sum = static_cast<RT*>(a.sum_out) + row * a.sum_stride;
  float s[NV][8], w1[8];  // w1: with one vector per thread the weights too are asked for before the reduction
  float2 sq2 = make_float2(0.f, 0.f);
  if constexpr (WIDE && NV == 1) {
    if (tid * 8 < a.H) load8_dt<true>(a.w, a.w_dtype, tid * 8, 8, w1);
  }
  if constexpr (WIDE) {
    // every load of the row is under way before the first is used
    constexpr int kX = sizeof(XT) / 2, kR = sizeof(RT) / 2;
    uint4 rx[NV][kX], rr[NV][kR];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * nt + tid) * 8;
#pragma unroll
      for (int k = 0; k < kX; ++k)
        rx[i][k] = c < a.H ? reinterpret_cast<const uint4*>(x + c)[k] : make_uint4(0, 0, 0, 0);
    }
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * nt + tid) * 8;
#pragma unroll
        for (int k = 0; k < kR; ++k)
          rr[i][k] = c < a.H ? reinterpret_cast<const uint4*>(res + c)[k] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float r[8];
        unpack8<XT>(rx[i], s[i]);
        unpack8<RT>(rr[i], r);
#pragma unroll
        for (int j = 0; j < 8; j += 2) add2(s[i] + j, make_float2(r[j], r[j + 1]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack8<XT>(rx[i], s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first_column<false>(i), n = a.H - c;
      load8<XT, false>(x + c, n, s[i]);
      if (a.residual) {
        float r[8];
        load8<RT, false>(res + c, n, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] += r[j];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first_column<WIDE>(i), n = a.H - c;
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      sq2 = fma2(make_float2(s[i][j], s[i][j + 1]), make_float2(s[i][j], s[i][j + 1]), sq2);
    if (a.sum_out && n > 0) store8<RT, WIDE>(sum + c, n, s[i]);
  }
  // z = (s * w) * r.  Rounding keeps order, so the row's largest |z| is that of |s * w|, times r: where the weights are
  // there in time, one reduction gives both.
  constexpr bool kEarly = WIDE && NV == 1;
  float sq = sq2.x + sq2.y, peak = 0.0f;  // peak: of the row, for the row-scaled outputs
  if constexpr (kEarly) {
    if (tid * 8 < a.H) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 z = mul2(make_float2(s[0][j], s[0][j + 1]), make_float2(w1[j] + a.w_offset, w1[j + 1] + a.w_offset));
        s[0][j] = z.x;
        s[0][j + 1] = z.y;
      }
    }
    if (per_row) {
#pragma unroll
      for (int j = 0; j < 8; ++j) peak = fmaxf(peak, fabsf(s[0][j]));
      block_reduce<true, true>(sq, peak, buf);
    } else {
      block_reduce<true, false>(sq, peak, buf);
    }
  } else {
    block_reduce<true, false>(sq, peak, buf);
  }
  const float mean = fmaf(sq, 1.0f / (float)a.H, a.eps);
  const float r = mean == 0.0f ? 0.0f : rsqrtf(mean);  // (eps = 0 and a row of zeros, or squares below fp32's range: z = 0)
  const bool fp8 = fmt == MOE_NORM_Q_E4M3_G128 || fmt == MOE_NORM_Q_E4M3_ROW;
  if (fp8 && r == 0.0f) {  // fp8 codes are taken before r: z = 0 has codes 0 too
    peak = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = 0.0f;
  }
  if (kEarly && !fp8) peak = fmaxf(peak * r, 0.0f);  // (no number: 0, as the maximum of the |z| would be)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first_column<WIDE>(i), n = a.H - c;
    if (n > 0) {
      float w[8];
      if constexpr (!kEarly) load8_dt<WIDE>(a.w, a.w_dtype, c, n, w);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float2 z = make_float2(s[i][j], s[i][j + 1]);
        if constexpr (!kEarly) z = mul2(z, make_float2(w[j] + a.w_offset, w[j + 1] + a.w_offset));
        if (!fp8) z = mul2(z, make_float2(r, r));
        s[i][j] = z.x;
        s[i][j + 1] = z.y;
      }
      if (a.y) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fp8 ? s[i][j] * r : s[i][j];
        store8_dt<WIDE>(a.y, a.y_dtype, row * a.y_stride + c, n, y);
      }
    }
    if (!kEarly && per_row) {
#pragma unroll
      for (int j = 0; j < 8; ++j) peak = fmaxf(peak, fabsf(s[i][j]));
    }
  }
  if (!kEarly && per_row) block_reduce<false, true>(sq, peak, buf);
  if constexpr (!WIDE) {
    if (fmt != MOE_NORM_Q_NONE) put_codes_narrow<NV>(a, row, s, peak, r);
  } else if constexpr (FMT != MOE_NORM_Q_NONE) {
    put_codes<NV, FMT>(a, row, s, peak, r);
  }
}

template <typename XT, typename RT, int NV, bool WIDE>
void launch_fmt(const NormArgs& a, int threads, cudaStream_t s) {
  const dim3 grid((unsigned)a.T);
  if constexpr (WIDE) {
    switch (a.q_fmt) {
      case MOE_NORM_Q_NONE: add_rmsnorm_kernel<XT, RT, NV, true, MOE_NORM_Q_NONE><<<grid, threads, 0, s>>>(a); break;
      case MOE_NORM_Q_Q8K: add_rmsnorm_kernel<XT, RT, NV, true, MOE_NORM_Q_Q8K><<<grid, threads, 0, s>>>(a); break;
      case MOE_NORM_Q_E4M3_G128:
        add_rmsnorm_kernel<XT, RT, NV, true, MOE_NORM_Q_E4M3_G128><<<grid, threads, 0, s>>>(a);
        break;
      case MOE_NORM_Q_E4M3_ROW:
        add_rmsnorm_kernel<XT, RT, NV, true, MOE_NORM_Q_E4M3_ROW><<<grid, threads, 0, s>>>(a);
        break;
      default: add_rmsnorm_kernel<XT, RT, NV, true, MOE_NORM_Q_INT8_ROW><<<grid, threads, 0, s>>>(a);
    }
  } else {
    add_rmsnorm_kernel<XT, RT, NV, false, -1><<<grid, threads, 0, s>>>(a);
  }
}

template <typename XT, typename RT, bool WIDE>
cudaError_t launch_nv(const NormArgs& a, cudaStream_t s) {
  const int vecs = (a.H + 7) / 8;
  // Few rows: latency counts, one vector per thread.  Many rows: two, so that a CTA's loads are larger and a
  // reduction is shared by more columns (8192 rows of 4096, fp8 codes: 37 us; with one vector 40, with four 39).
  // Rows of more than 8192 columns: four.
  int nv = a.T > 2 * num_sms() ? 2 : 1;
  while (nv < 4 && vecs > (nv == 1 ? 1024 : 512) * nv) nv *= 2;
  const int threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
  note_launch();
  if (nv == 1) launch_fmt<XT, RT, 1, WIDE>(a, threads, s);
  else if (nv == 2) launch_fmt<XT, RT, 2, WIDE>(a, threads, s);
  else launch_fmt<XT, RT, 4, WIDE>(a, threads, s);
  return cudaGetLastError();
}

template <typename XT, typename RT>
cudaError_t launch_types(const NormArgs& a, cudaStream_t s) {
  return a.wide ? launch_nv<XT, RT, true>(a, s) : launch_nv<XT, RT, false>(a, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (a.x_dtype == MOE_DT_F32) return launch_types<float, float>(a, s);
  if (a.x_dtype == MOE_DT_BF16)
    return a.r_dtype == MOE_DT_F32 ? launch_types<__nv_bfloat16, float>(a, s)
                                   : launch_types<__nv_bfloat16, __nv_bfloat16>(a, s);
  return a.r_dtype == MOE_DT_F32 ? launch_types<__half, float>(a, s) : launch_types<__half, __half>(a, s);
}

}  // namespace moe
