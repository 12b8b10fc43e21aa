// The paged cache in 8 bits: quantising a chunk's keys and values as they are
// written, and reading sequences back.
//
//   d = max|x| / top,  code = x / d;      x' = code * d
//
// What bounds both: memory, and for a decode step latency.  Every element is
// read once and written once.  Appending takes a warp per token and few heads: a
// head's D elements are 8 to a lane, so its maximum is a few shuffles among a
// group of lanes (keys and values together, a half of a register each), and all
// of a warp's loads are under way before the token's page is looked up.  Reading
// back takes 16 codes to a lane, as many lanes to a row as it has of them, up to
// a warp.
//
// What it measured: 5257 tokens of 8 heads of 128 (bf16 to e4m3) appended in 9.3
// us, 3.5 TB/s, two rounds of CTAs whose warps wait for their loads and then
// divide (a warp for all 8 heads of a token: 2 us more); 64 tokens of 4 heads 2.2.
// Up to 32768 keys of each of three sequences, 8 heads of 128, e4m3 to bf16, read
// back in 71 us, 5.8 TB/s (four rows of a warp at a time: 83 us).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "moe_kv.cuh"
#include "moe_overlap.cuh"
#include "moe_q8.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float2 pair_f(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// 8 elements of 16 bits, in pairs
template <bool WIDE>
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  if constexpr (WIDE) {
    return *reinterpret_cast<const uint4*>(p);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A vector's scale from its largest magnitude, the bits of a 16-bit number.
template <bool BF16, int FMT>
__device__ __forceinline__ float scale_of(uint32_t peak) {
  constexpr float kTop = FMT == MOE_DT_E4M3 ? 448.0f : 127.0f, kPart = 1.0f / kTop;
  const float x = pair_f(peak, BF16).x, q = x * kPart;
  const float d = fmaxf(x < 1e-25f ? x / kTop : fmaf(fmaf(-q, kTop, x), kPart, q), 1.17549435e-38f);  // (as codes_of divides)
  return peak >= (BF16 ? 0x7f80u : 0x7c00u) ? __uint_as_float(0x7fc00000u) : peak == 0 ? 0.0f : d;
}
// Codes of 8 elements x / d.  The quotient is rounded as IEEE division rounds it, by Markstein's theorem (IBM J. Res.
// Dev. 34, 1990): with the correctly rounded reciprocal r and the exact remainder of q = x r, q + r (x - q d) in fused
// operations.  The remainder is exact while it is a normal number or 0; tiny scales take the division itself.
template <bool BF16, int FMT>
__device__ __forceinline__ uint2 codes_of(uint4 x, float d) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float2 z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = pair_f(w[i], BF16);
  if (d >= 1e-28f) {
    const float r = __frcp_rn(d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float q0 = z[i].x * r, q1 = z[i].y * r;
      z[i].x = fmaf(fmaf(-q0, d, z[i].x), r, q0);
      z[i].y = fmaf(fmaf(-q1, d, z[i].y), r, q1);
    }
  } else if (d > 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i].x /= d, z[i].y /= d;
  } else {  // zeros, or not finite
    return make_uint2(0, 0);
  }
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (FMT == MOE_DT_E4M3) {
      code[i] = __nv_cvt_float2_to_fp8x2(z[i], __NV_SATFINITE, __NV_E4M3);
    } else {
      const int a = (int)roundf(z[i].x), b = (int)roundf(z[i].y);  // |z| < 127.5: the scale is off by half a step at most
      code[i] = (uint32_t)(a & 0xff) | (uint32_t)(b & 0xff) << 8;
    }
  }
  uint2 c = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
  if constexpr (FMT == MOE_DT_E4M3) {  // the sign of a zero, which the corrected quotient has lost
    c.x |= __byte_perm(w[0], w[1], 0x7531) & 0x80808080u;
    c.y |= __byte_perm(w[2], w[3], 0x7531) & 0x80808080u;
  }
  return c;
}
__device__ __forceinline__ uint32_t peak_of(uint4 x) {  // in two halves; magnitudes of 16-bit numbers order as integers
  return __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
}

template <bool WIDE>
__device__ __forceinline__ void store_codes(uint8_t* p, uint2 c) {
  if constexpr (WIDE) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = (uint8_t)(c.x >> 8 * i), p[4 + i] = (uint8_t)(c.y >> 8 * i);
  }
}

// kBatch: loads of a lane that are under way at one time, of keys and of values each.  kWidth: lanes of a head (0: any).
template <bool BF16, int FMT, bool WIDE, int kBatch, int kWidth>
__global__ void __launch_bounds__(128) append_kernel(const KvAppendQ8Args g) {
  const KvAppendArgs& a = g.a;
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  int width = kWidth;
  if constexpr (kWidth == 0) {
    width = 1;
    while (width < a.kv.D / 8) width *= 2;
  }
  const int per = 32 / width, group = lane / width, c = (lane - group * width) * 8;
  const int h0 = blockIdx.y * kBatch * per + group;  // the warp's first heads, and per more for each of its loads
  const bool in_row = c < a.kv.D;
  const uint16_t* k = static_cast<const uint16_t*>(a.k) + (int64_t)t * a.k_stride + h0 * a.k_head_stride + c;
  const uint16_t* v = static_cast<const uint16_t*>(a.v) + (int64_t)t * a.v_stride + h0 * a.v_head_stride + c;
  uint4 kb[kBatch], vb[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int h = h0 + u * per;
    kb[u] = vb[u] = make_uint4(0, 0, 0, 0);
    if (h < a.kv.Hkv && in_row) {
      kb[u] = load8<WIDE>(k + u * per * a.k_head_stride);
      vb[u] = load8<WIDE>(v + u * per * a.v_head_stride);
    }
  }
  const int b = find_seq(a.cu_q, a.kv.n_seqs, t, lane);
  const SeqInfo s = seq_info(a.kv, a.cu_q, a.kv_len, a.T, b);
  if (!s.ok) {
    if (lane == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  if (t < s.q0 || t >= s.q0 + s.n) return;  // a row that belongs to no sequence
  const int pos = s.kv - s.n + (t - s.q0);
  const int page = pos >= 0 ? __ldg(a.table + (int64_t)b * a.kv.table_stride + pos / a.kv.page_size) : -1;
  if (page < 0 || page >= a.kv.num_pages) {
    if (lane == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  const int slot = pos % a.kv.page_size;
  uint8_t* kc = static_cast<uint8_t*>(a.k_cache) + (int64_t)page * a.kv.k_page_stride + slot * a.kv.k_row_stride +
                h0 * a.kv.k_head_stride + c;
  uint8_t* vc = static_cast<uint8_t*>(a.v_cache) + (int64_t)page * a.kv.v_page_stride + slot * a.kv.v_row_stride +
                h0 * a.kv.v_head_stride + c;
  float* ks = g.sc.k + (int64_t)page * g.sc.k_page_stride + slot * g.sc.k_row_stride + h0 * g.sc.k_head_stride;
  float* vs = g.sc.v + (int64_t)page * g.sc.v_page_stride + slot * g.sc.v_row_stride + h0 * g.sc.v_head_stride;
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int h = h0 + u * per;
    // the largest of the key and of the value, a half each, over the lanes that hold them
    const uint32_t kp = peak_of(kb[u]), vp = peak_of(vb[u]);
    uint32_t m = max(kp & 0xffffu, kp >> 16) | max(vp & 0xffffu, vp >> 16) << 16;
#pragma unroll
    for (int o = (kWidth ? kWidth : width) >> 1; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float kd = scale_of<BF16, FMT>(m & 0xffffu), vd = scale_of<BF16, FMT>(m >> 16);
    const uint2 kq = codes_of<BF16, FMT>(kb[u], kd), vq = codes_of<BF16, FMT>(vb[u], vd);
    if (h < a.kv.Hkv && in_row) {
      store_codes<WIDE>(kc + u * per * a.kv.k_head_stride, kq);
      store_codes<WIDE>(vc + u * per * a.kv.v_head_stride, vq);
      if (c == 0) {
        ks[u * per * g.sc.k_head_stride] = kd;
        vs[u * per * g.sc.v_head_stride] = vd;
      }
    }
  }
}

template <int OUT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (OUT == MOE_DT_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// N codes times their scale to N elements of type OUT: an fp32 product, rounded again where OUT is narrower
template <int FMT, int OUT, int N, bool WIDE>
__device__ __forceinline__ void put_values(const uint32_t* w, float d, void* out, int64_t at) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) four_values<FMT>(w[i], v + 4 * i);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= d;
  if constexpr (OUT == MOE_DT_F32) {
    float* p = static_cast<float*>(out) + at;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      if constexpr (WIDE) reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      else p[4 * i] = v[4 * i], p[4 * i + 1] = v[4 * i + 1], p[4 * i + 2] = v[4 * i + 2], p[4 * i + 3] = v[4 * i + 3];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(out) + at;
    uint32_t r[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) r[i] = pack16<OUT>(v[2 * i], v[2 * i + 1]);
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) p[2 * i] = (uint16_t)r[i], p[2 * i + 1] = (uint16_t)(r[i] >> 16);
    }
  }
}
template <int N, bool WIDE>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t* w) {
  if constexpr (WIDE) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = (uint32_t)p[4 * i] | (uint32_t)p[4 * i + 1] << 8 | (uint32_t)p[4 * i + 2] << 16 | (uint32_t)p[4 * i + 3] << 24;
  }
}

// A row is the work of 2^shift lanes of a warp: 32, or as many as it has pieces of N codes.
template <int FMT, int OUT, bool WIDE>
__global__ void __launch_bounds__(128) read_kernel(const KvReadQ8Args a, int shift) {
  constexpr int N = WIDE ? 16 : 8;
  let_next_start();
  wait_for_previous();
  if (blockIdx.x == 0) {  // every sequence's rows: in range, and before the next one's
    for (int b = threadIdx.x; b < a.kv.n_seqs; b += blockDim.x) {
      const int64_t len = __ldg(a.kv_len + b), at = __ldg(a.first + b);
      const int64_t end = b + 1 < a.kv.n_seqs ? min(__ldg(a.first + b + 1), a.rows) : a.rows;
      if (len < 0 || len > (int64_t)a.kv.max_pages * a.kv.page_size || (len > 0 && (at < 0 || at + len > end)))
        set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    }
  }
  const int width = 1 << shift, lane = threadIdx.x & (width - 1);
  const int64_t r = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> shift;
  if (r >= a.rows) return;
  int b = 0;  // the last sequence that starts at or before the row
  for (int n = a.kv.n_seqs; n > 1;) {
    const int half = n / 2;
    if (__ldg(a.first + b + half) <= r) b += half, n -= half;
    else n = half;
  }
  const int len = __ldg(a.kv_len + b);
  const int64_t j64 = r - __ldg(a.first + b);
  if (len > (int64_t)a.kv.max_pages * a.kv.page_size || j64 < 0 || j64 >= len) return;
  const int j = (int)j64, slot = j % a.kv.page_size;
  const int page = __ldg(a.table + (int64_t)b * a.kv.table_stride + j / a.kv.page_size);
  if (page < 0 || page >= a.kv.num_pages) {
    if (lane == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  const uint8_t* kc = static_cast<const uint8_t*>(a.k_cache) + (int64_t)page * a.kv.k_page_stride + slot * a.kv.k_row_stride;
  const uint8_t* vc = static_cast<const uint8_t*>(a.v_cache) + (int64_t)page * a.kv.v_page_stride + slot * a.kv.v_row_stride;
  const float* ks = a.sc.k + (int64_t)page * a.sc.k_page_stride + slot * a.sc.k_row_stride;
  const float* vs = a.sc.v + (int64_t)page * a.sc.v_page_stride + slot * a.sc.v_row_stride;
  const int vecs = a.kv.D / N, total = a.kv.Hkv * vecs;
  for (int i = lane; i < total; i += width) {
    const int h = i / vecs, c = (i - h * vecs) * N;
    uint32_t kw[N / 4], vw[N / 4];
    load_codes<N, WIDE>(kc + h * a.kv.k_head_stride + c, kw);
    load_codes<N, WIDE>(vc + h * a.kv.v_head_stride + c, vw);
    const float kd = ks[h * a.sc.k_head_stride], vd = vs[h * a.sc.v_head_stride];
    put_values<FMT, OUT, N, WIDE>(kw, kd, a.k_out, r * a.k_stride + h * a.k_head_stride + c);
    put_values<FMT, OUT, N, WIDE>(vw, vd, a.v_out, r * a.v_stride + h * a.v_head_stride + c);
  }
}

template <bool BF16, int FMT, int kBatch>
cudaError_t append_as(const KvAppendQ8Args& a, int warps, cudaStream_t s) {
  int width = 1;  // lanes of a head
  while (width < a.a.kv.D / 8) width *= 2;
  const int heads = kBatch * (32 / width);  // of a warp
  const dim3 grid((unsigned)((a.a.T + warps - 1) / warps), (unsigned)((a.a.kv.Hkv + heads - 1) / heads));
  // The usual head sizes, 64, 128 and 256, and all that need as many lanes, have their count of lanes in the code: with
  // it, and with the scales' quotients as those of the elements, 9.3 us where the other form took 10.3 (5257 tokens).
  const auto run = [&](auto kern) { return launch_overlapping(kern, grid, 32 * warps, 0, 1, s, a); };
  if (!a.a.wide) return run(append_kernel<BF16, FMT, false, kBatch, 0>);
  switch (width) {
    case 8: return run(append_kernel<BF16, FMT, true, kBatch, 8>);
    case 16: return run(append_kernel<BF16, FMT, true, kBatch, 16>);
    case 32: return run(append_kernel<BF16, FMT, true, kBatch, 32>);
    default: return run(append_kernel<BF16, FMT, true, kBatch, 0>);
  }
}
template <bool BF16, int FMT>
cudaError_t append(const KvAppendQ8Args& a, cudaStream_t s) {
  // Few tokens are latency: a warp to each token and as few heads as it holds.  Many share the way to their page among the
  // heads of two loads.  In us with one / two, bf16 to e4m3, tokens one after the other in a sequence:
  //                      64           304          456          608          1000         1500         5257
  //   4 heads of 128     1.9 / 2.3    2.0 / 2.3    2.2 / 2.3    2.5 / 2.3    3.1 / 3.4    3.4 / 4.2    11.1 / 4.9
  //   8 heads of 128     1.9 / 2.3    2.5 / 2.4    3.0 / 2.5    2.9 / 3.6    4.4 / 4.5    6.4 / 4.7    21.6 / 8.8
  //   2 heads of 256     2.0 / 2.3    2.0 / 2.4    2.3 / 2.4    2.6 / 2.4    3.2 / 3.4    3.4 / 4.2    11.1 / 5.0
  return a.a.T <= 4 * num_sms() ? append_as<BF16, FMT, 1>(a, 1, s) : append_as<BF16, FMT, 2>(a, 4, s);
}
template <int FMT, int OUT>
cudaError_t read(const KvReadQ8Args& a, cudaStream_t s) {
  const int pieces = a.kv.Hkv * a.kv.D / (a.wide ? 16 : 8);
  int shift = 0;
  while (shift < 5 && 1 << shift < pieces) ++shift;
  const unsigned grid = (unsigned)std::max<int64_t>(1, (((int64_t)a.rows << shift) + 127) / 128);  // (the first looks at the lengths)
  return launch_overlapping(a.wide ? read_kernel<FMT, OUT, true> : read_kernel<FMT, OUT, false>, dim3(grid), 128, 0, 1, s, a, shift);
}
template <int FMT>
cudaError_t read_as(const KvReadQ8Args& a, cudaStream_t s) {
  if (a.out_dtype == MOE_DT_F32) return read<FMT, MOE_DT_F32>(a, s);
  return a.out_dtype == MOE_DT_BF16 ? read<FMT, MOE_DT_BF16>(a, s) : read<FMT, MOE_DT_F16>(a, s);
}

}  // namespace

cudaError_t launch_kv_append_q8(const KvAppendQ8Args& a, cudaStream_t s) {
  if (a.a.T == 0) return cudaSuccess;
  const bool bf16 = a.x_dtype == MOE_DT_BF16, e4m3 = a.a.kv.dtype == MOE_DT_E4M3;
  note_launch();
  if (bf16) return e4m3 ? append<true, MOE_DT_E4M3>(a, s) : append<true, MOE_DT_INT8>(a, s);
  return e4m3 ? append<false, MOE_DT_E4M3>(a, s) : append<false, MOE_DT_INT8>(a, s);
}

cudaError_t launch_kv_read_q8(const KvReadQ8Args& a, cudaStream_t s) {
  note_launch();
  return a.kv.dtype == MOE_DT_E4M3 ? read_as<MOE_DT_E4M3>(a, s) : read_as<MOE_DT_INT8>(a, s);
}

}  // namespace moe
