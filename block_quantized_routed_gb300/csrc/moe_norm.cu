// Residual addition, root-mean-square norm and an 8-bit output in one pass.
//
//   s = x + residual,  z = s * rsqrt(mean(s^2) + eps) * (w + offset)
//   q = codes of z with one scale per 256 / 128 columns or per row
//
// What bounds it: memory.  Every element of x and residual is read once and
// every output written once; s stays in registers between the sum of squares
// and the scaling, so there is no second pass over global memory.
//
// Layout: one CTA per row.  A thread holds NV vectors of 8 consecutive
// columns (vector i * blockDim + tid), so a warp's vectors are 256
// consecutive columns: a q8_K block is one warp-wide maximum, a group of 128
// columns a half-warp's, and neither needs shared memory.  Rows that are not
// 16-byte aligned (odd H, odd strides) run the same mapping with element-wise
// guarded loads (WIDE = false).
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "moe_device.cuh"
#include "moe_internal.h"

#ifndef MOE_NORM_THREADS
#define MOE_NORM_THREADS 1024
#endif
#ifndef MOE_NORM_STAGES
#define MOE_NORM_STAGES 3
#endif
#ifndef MOE_NORM_NV
#define MOE_NORM_NV 2
#endif

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

// 8 consecutive elements as fp32; `n` of them exist (WIDE: all 8, 16-byte aligned)
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
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f<T>(p[i]) : 0.0f;
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

template <typename T, bool WIDE>
__device__ __forceinline__ void store8(T* p, int n, const float* v) {
  if constexpr (WIDE) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      T e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = from_f<T>(v[i]);
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f<T>(v[i]);
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

// all threads of the block get the sum / the maximum, in a fixed order
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = lane < nw ? buf[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  return v;
}

// The q8_K rounding of z / d: half away from zero, clamped.  The product with
// the reciprocal is within 2 ulp of the IEEE quotient (at most 127: 2^-16), so
// both round alike unless it is that near a half; only there it is divided.
__device__ __forceinline__ int q8k_code(float z, float d, float inv) {
  float x = z * inv;
  if (fabsf(fabsf(x - truncf(x)) - 0.5f) < 3.1e-5f) x = __fdiv_rn(z, d);
  return (int)fminf(127.0f, fmaxf(-127.0f, roundf(x)));
}

// Scales z (s[NV][8]) into y and the 8-bit output of one row; `peak` is the
// thread's largest |z| (row-scaled outputs only), buf one block_reduce buffer.
template <int NV, bool WIDE>
__device__ __forceinline__ void put_codes(const NormArgs& a, int64_t row, float (&s)[NV][8], float peak, float* buf) {
  const int tid = threadIdx.x, nt = blockDim.x;
  const bool per_row = a.q_fmt == MOE_NORM_Q_E4M3_ROW || a.q_fmt == MOE_NORM_Q_INT8_ROW;
  const bool fp8 = a.q_fmt == MOE_NORM_Q_E4M3_G128 || a.q_fmt == MOE_NORM_Q_E4M3_ROW;
  const float top = fp8 ? 448.0f : 127.0f;
  float d = 0.0f;
  if (per_row) {
    peak = block_reduce<true>(peak, buf);
    d = __fdiv_rn(peak, top);
    if (tid == 0) a.d[row] = d;
  }
  const int group = a.q_fmt == MOE_NORM_Q_Q8K ? 256 : 128;
  const int groups = (a.H + group - 1) / group;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + tid) * 8, n = a.H - c;
    if (!per_row) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(s[i][j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (group == 256) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      d = __fdiv_rn(m, top);
      if (n > 0 && c % group == 0) a.d[row * groups + c / group] = d;
    }
    // d = 0 only where every z of the group is 0 (or too small for its quotient to exist).  A reciprocal beyond
    // fp32 (d below 2^-127) is not used: such groups are divided.
    float inv = d > 0.0f ? 1.0f / d : 0.0f, dq = d;
    if (inv > 3e38f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = __fdiv_rn(s[i][j], d);
      inv = dq = 1.0f;
    }
    uint8_t q[8];
    int sum = 0;
    if (fp8) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        *reinterpret_cast<__nv_fp8x2_storage_t*>(q + j) = __nv_cvt_float2_to_fp8x2(
            make_float2(s[i][j] * inv, s[i][j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int code = q8k_code(s[i][j], dq, inv);
        q[j] = (uint8_t)(int8_t)code;
        sum += code;
      }
    }
    uint8_t* out = static_cast<uint8_t*>(a.q) + row * a.H + c;
    if constexpr (WIDE) {
      if (n > 0) *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(q);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) out[j] = q[j];
    }
    if (a.bsum16) {  // q8_K: two lanes hold the 16 codes
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      if (n > 0 && (tid & 1) == 0) a.bsum16[row * (a.H / 16) + c / 16] = (int16_t)sum;
    }
  }
}

template <typename XT, typename RT, int NV, bool WIDE>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const NormArgs a) {
  __shared__ float buf[2][32];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x;
  const XT* x = static_cast<const XT*>(a.x) + row * a.x_stride;
  const RT* res = static_cast<const RT*>(a.residual) + row * a.r_stride;
  float s[NV][8];
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + tid) * 8, n = a.H - c;
    if (n > 0) {
      load8<XT, WIDE>(x + c, n, s[i]);
      if (a.residual) {
        float r[8];
        load8<RT, WIDE>(res + c, n, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + tid) * 8, n = a.H - c;
#pragma unroll
    for (int j = 0; j < 8; ++j) sq = fmaf(s[i][j], s[i][j], sq);
    if (a.sum_out && n > 0) store8<RT, WIDE>(static_cast<RT*>(a.sum_out) + row * a.sum_stride + c, n, s[i]);
  }
  sq = block_reduce<false>(sq, buf[0]);
  const float r = 1.0f / sqrtf(sq / (float)a.H + a.eps);
  const bool per_row = a.q_fmt == MOE_NORM_Q_E4M3_ROW || a.q_fmt == MOE_NORM_Q_INT8_ROW;
  float peak = 0.0f;  // of the row, for the row-scaled outputs
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + tid) * 8, n = a.H - c;
    float w[8];
    if (n > 0) {
      load8_dt<WIDE>(a.w, a.w_dtype, c, n, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = s[i][j] * r * (w[j] + a.w_offset);
      if (a.y) store8_dt<WIDE>(a.y, a.y_dtype, row * a.y_stride + c, n, s[i]);
    }
    if (per_row) {
#pragma unroll
      for (int j = 0; j < 8; ++j) peak = fmaxf(peak, fabsf(s[i][j]));
    }
  }
  if (a.q_fmt == MOE_NORM_Q_NONE) return;
  put_codes<NV, WIDE>(a, row, s, peak, buf[1]);
}

// The same for many rows: a CTA stays on its SM and walks the rows.  The
// weights are kept in registers; the rows ahead come by asynchronous copies
// into shared memory, where each thread reads back only what it asked for
// itself (no barrier), so the loads of the next rows are under way through
// both reductions of this one.
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
template <typename T>
__device__ __forceinline__ void copy8(uint4* dst, const T* src) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst + i)),
                 "l"(reinterpret_cast<const uint4*>(src) + i)
                 : "memory");
}

template <typename XT, typename RT>
constexpr int row_vec_bytes() { return 8 * (int)(sizeof(XT) + sizeof(RT)); }  // x and residual of one vector

template <typename XT, typename RT, int NV, int STAGES>
__global__ void __launch_bounds__(512, NV > 2 ? 1 : 2) add_rmsnorm_rows_kernel(const NormArgs a) {
  __shared__ float buf[2][2][32];
  extern __shared__ uint4 ring[];  // [stage][vector][x | residual][thread]
  constexpr int kX = sizeof(XT) / 2, kR = sizeof(RT) / 2;
  const int tid = threadIdx.x, nt = blockDim.x;
  const bool per_row = a.q_fmt == MOE_NORM_Q_E4M3_ROW || a.q_fmt == MOE_NORM_Q_INT8_ROW;
  const bool res = a.residual != nullptr;
  const auto slot = [&](int stage, int i) { return ring + ((size_t)(stage * NV + i) * nt + tid) * (kX + kR); };
  const auto fetch = [&](int64_t r, int stage) {
    if (r < a.T) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * nt + tid) * 8;
        if (c < a.H) {
          copy8<XT>(slot(stage, i), static_cast<const XT*>(a.x) + r * a.x_stride + c);
          if (res) copy8<RT>(slot(stage, i) + kX, static_cast<const RT*>(a.residual) + r * a.r_stride + c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t row = blockIdx.x;
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) fetch(row + (int64_t)k * gridDim.x, k);
  float w[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + tid) * 8;
    if (c < a.H) {
      load8_dt<true>(a.w, a.w_dtype, c, 8, w[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] += a.w_offset;
    }
  }
  int stage = 0;
  for (int odd = 0; row < a.T; row += gridDim.x, odd ^= 1) {
    fetch(row + (int64_t)(STAGES - 1) * gridDim.x, stage == 0 ? STAGES - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    float s[NV][8];
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * nt + tid) * 8;
      if (c < a.H) {
        unpack8<XT>(slot(stage, i), s[i]);
        if (res) {
          float r[8];
          unpack8<RT>(slot(stage, i) + kX, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[i][j] += r[j];
        }
        if (a.sum_out) store8<RT, true>(static_cast<RT*>(a.sum_out) + row * a.sum_stride + c, 8, s[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(s[i][j], s[i][j], sq);
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
    sq = block_reduce<false>(sq, buf[odd][0]);
    const float r = 1.0f / sqrtf(sq / (float)a.H + a.eps);
    float peak = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * nt + tid) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = c < a.H ? s[i][j] * r * w[i][j] : 0.0f;
      if (a.y && c < a.H) store8_dt<true>(a.y, a.y_dtype, row * a.y_stride + c, 8, s[i]);
      if (per_row) {
#pragma unroll
        for (int j = 0; j < 8; ++j) peak = fmaxf(peak, fabsf(s[i][j]));
      }
    }
    if (a.q_fmt != MOE_NORM_Q_NONE) put_codes<NV, true>(a, row, s, peak, buf[odd][1]);
  }
}

template <typename XT, typename RT, int NV>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t s) {
  constexpr int kStages = MOE_NORM_STAGES;
  const int vecs = a.H / 8, threads = ((vecs + NV - 1) / NV + 31) / 32 * 32;
  const int smem = kStages * NV * threads * row_vec_bytes<XT, RT>();
  auto kern = add_rmsnorm_rows_kernel<XT, RT, NV, kStages>;
  static bool opted = false;
  if (!opted) {
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (err != cudaSuccess) return err;
    opted = true;
  }
  const int per_sm = std::max(1, std::min(MOE_NORM_THREADS / threads, 220 * 1024 / (smem + 2048)));
  const unsigned grid = (unsigned)std::min<int64_t>(a.T, (int64_t)num_sms() * per_sm);
  note_launch();
  kern<<<grid, threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename XT, typename RT, bool WIDE>
cudaError_t launch_nv(const NormArgs& a, cudaStream_t s) {
  const int vecs = (a.H + 7) / 8;
  if constexpr (WIDE) {
    // rows of up to 64 KB in, three of which fit an SM's shared memory
    if (a.T >= 8 * num_sms() && a.H / 8 * row_vec_bytes<XT, RT>() <= 64 * 1024)
      return vecs <= 1024 ? launch_rows<XT, RT, MOE_NORM_NV>(a, s) : launch_rows<XT, RT, 4>(a, s);
  }
  // Few rows: latency counts, one vector per thread.  Many rows: two to eight
  // vectors per thread, so that a CTA is small and its loads are in flight together.
  int nv = 1;
  if (a.T > 2 * num_sms())
    while (nv < 4 && vecs > 128 * nv) nv *= 2;
  while (nv < 8 && vecs > 1024 * nv) nv *= 2;
  const int threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
  note_launch();
  const dim3 grid((unsigned)a.T);
  switch (nv) {
    case 1: add_rmsnorm_kernel<XT, RT, 1, WIDE><<<grid, threads, 0, s>>>(a); break;
    case 2: add_rmsnorm_kernel<XT, RT, 2, WIDE><<<grid, threads, 0, s>>>(a); break;
    default: add_rmsnorm_kernel<XT, RT, 4, WIDE><<<grid, threads, 0, s>>>(a); break;
  }
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
