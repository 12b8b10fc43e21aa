// The paged cache in 8 bits: quantising a chunk's keys and values as they are
// written, and reading sequences back.
//
//   d = max|x| / top,  code = x / d;      x' = code * d
//
// What bounds both: memory, and for a decode step latency.  Every element is
// read once and written once.  Appending takes one warp per token: a head's D
// elements are 8 to a lane, so its maximum is a few shuffles among a group of
// lanes, and several heads' keys and values are in flight before the token's
// page is looked up.  Reading back takes one warp per row, 16 codes to a lane.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "moe_kv.cuh"
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
  if constexpr (WIDE) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes and scale of a vector whose elements are spread over `width` lanes (a power of two), 8 each.
template <bool BF16, int FMT>
__device__ __forceinline__ uint2 quantise(uint4 x, int width, float& d) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  // magnitudes of 16-bit numbers order as integers, infinities and NaN last
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  m = max(m & 0xffffu, m >> 16);
  for (int o = width >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m >= (BF16 ? 0x7f80u : 0x7c00u)) {
    d = __uint_as_float(0x7fc00000u);
    return make_uint2(0, 0);
  }
  if (m == 0) {
    d = 0.0f;
    return make_uint2(0, 0);
  }
  d = fmaxf(pair_f(m, BF16).x / (FMT == MOE_DT_E4M3 ? 448.0f : 127.0f), 1.17549435e-38f);
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 z = pair_f(w[i], BF16);
    z.x /= d;
    z.y /= d;
    if constexpr (FMT == MOE_DT_E4M3) {
      code[i] = __nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E4M3);
    } else {
      const int a = (int)fminf(127.0f, fmaxf(-127.0f, roundf(z.x))), b = (int)fminf(127.0f, fmaxf(-127.0f, roundf(z.y)));
      code[i] = (uint32_t)(a & 0xff) | (uint32_t)(b & 0xff) << 8;
    }
  }
  return make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
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

template <bool BF16, int FMT, bool WIDE>
__global__ void __launch_bounds__(128) append_kernel(const KvAppendQ8Args g) {
  const KvAppendArgs& a = g.a;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  constexpr int kBatch = 4;
  const int vecs = a.kv.D / 8;  // 1 .. 32 of a head
  int width = 1;
  while (width < vecs) width *= 2;
  const int per = 32 / width, h0 = lane / width, c = (lane - h0 * width) * 8;
  const bool in_row = c < a.kv.D;
  const uint16_t* k = static_cast<const uint16_t*>(a.k) + (int64_t)t * a.k_stride;
  const uint16_t* v = static_cast<const uint16_t*>(a.v) + (int64_t)t * a.v_stride;
  uint4 kb[kBatch], vb[kBatch];
  const auto load = [&](int first) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = first + u * per + h0;
      kb[u] = vb[u] = make_uint4(0, 0, 0, 0);
      if (h < a.kv.Hkv && in_row) {
        kb[u] = load8<WIDE>(k + h * a.k_head_stride + c);
        vb[u] = load8<WIDE>(v + h * a.v_head_stride + c);
      }
    }
  };
  load(0);
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
  uint8_t* kc = static_cast<uint8_t*>(a.k_cache) + (int64_t)page * a.kv.k_page_stride + slot * a.kv.k_row_stride;
  uint8_t* vc = static_cast<uint8_t*>(a.v_cache) + (int64_t)page * a.kv.v_page_stride + slot * a.kv.v_row_stride;
  float* ks = g.sc.k + (int64_t)page * g.sc.k_page_stride + slot * g.sc.k_row_stride;
  float* vs = g.sc.v + (int64_t)page * g.sc.v_page_stride + slot * g.sc.v_row_stride;
  for (int first = 0; first < a.kv.Hkv; first += kBatch * per) {
    if (first) load(first);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (first + u * per >= a.kv.Hkv) break;  // the same for the whole warp
      const int h = first + u * per + h0;
      float kd, vd;
      const uint2 kq = quantise<BF16, FMT>(kb[u], width, kd), vq = quantise<BF16, FMT>(vb[u], width, vd);
      if (h < a.kv.Hkv && in_row) {
        store_codes<WIDE>(kc + h * a.kv.k_head_stride + c, kq);
        store_codes<WIDE>(vc + h * a.kv.v_head_stride + c, vq);
        if (c == 0) {
          ks[h * g.sc.k_head_stride] = kd;
          vs[h * g.sc.v_head_stride] = vd;
        }
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

// N codes times their scale to N elements of type OUT
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

template <int FMT, int OUT, bool WIDE>
__global__ void __launch_bounds__(128) read_kernel(const KvReadQ8Args a) {
  constexpr int N = WIDE ? 16 : 8;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) {  // every sequence's rows: in range, and before the next one's
    for (int b = threadIdx.x; b < a.kv.n_seqs; b += blockDim.x) {
      const int64_t len = __ldg(a.kv_len + b), at = __ldg(a.first + b);
      const int64_t end = b + 1 < a.kv.n_seqs ? min(__ldg(a.first + b + 1), a.rows) : a.rows;
      if (len < 0 || len > (int64_t)a.kv.max_pages * a.kv.page_size || (len > 0 && (at < 0 || at + len > end)))
        set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    }
  }
  const int r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (r >= a.rows) return;
  const int b = find_seq(a.first, a.kv.n_seqs, r, lane);
  const int len = __ldg(a.kv_len + b);
  const int64_t j64 = (int64_t)r - __ldg(a.first + b);
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
  constexpr int kBatch = 2;
  for (int i0 = lane; i0 < total; i0 += 32 * kBatch) {
    uint32_t kw[kBatch][N / 4], vw[kBatch][N / 4];
    float kd[kBatch], vd[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + 32 * u;
      if (i < total) {
        const int h = i / vecs, c = (i - h * vecs) * N;
        load_codes<N, WIDE>(kc + h * a.kv.k_head_stride + c, kw[u]);
        load_codes<N, WIDE>(vc + h * a.kv.v_head_stride + c, vw[u]);
        kd[u] = ks[h * a.sc.k_head_stride];
        vd[u] = vs[h * a.sc.v_head_stride];
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + 32 * u;
      if (i < total) {
        const int h = i / vecs, c = (i - h * vecs) * N;
        put_values<FMT, OUT, N, WIDE>(kw[u], kd[u], a.k_out, r * a.k_stride + h * a.k_head_stride + c);
        put_values<FMT, OUT, N, WIDE>(vw[u], vd[u], a.v_out, r * a.v_stride + h * a.v_head_stride + c);
      }
    }
  }
}

template <bool BF16, int FMT>
void append(const KvAppendQ8Args& a, unsigned grid, int threads, cudaStream_t s) {
  if (a.a.wide) append_kernel<BF16, FMT, true><<<grid, threads, 0, s>>>(a);
  else append_kernel<BF16, FMT, false><<<grid, threads, 0, s>>>(a);
}
template <int FMT, int OUT>
void read(const KvReadQ8Args& a, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.rows + 3) / 4);
  if (a.wide) read_kernel<FMT, OUT, true><<<grid, 128, 0, s>>>(a);
  else read_kernel<FMT, OUT, false><<<grid, 128, 0, s>>>(a);
}
template <int FMT>
void read_as(const KvReadQ8Args& a, cudaStream_t s) {
  if (a.out_dtype == MOE_DT_F32) read<FMT, MOE_DT_F32>(a, s);
  else if (a.out_dtype == MOE_DT_BF16) read<FMT, MOE_DT_BF16>(a, s);
  else read<FMT, MOE_DT_F16>(a, s);
}

}  // namespace

cudaError_t launch_kv_append_q8(const KvAppendQ8Args& a, cudaStream_t s) {
  if (a.a.T == 0) return cudaSuccess;
  const int warps = a.a.T <= 4 * num_sms() ? 1 : 4;
  const unsigned grid = (unsigned)((a.a.T + warps - 1) / warps);
  const bool bf16 = a.x_dtype == MOE_DT_BF16, e4m3 = a.a.kv.dtype == MOE_DT_E4M3;
  note_launch();
  if (bf16) e4m3 ? append<true, MOE_DT_E4M3>(a, grid, 32 * warps, s) : append<true, MOE_DT_INT8>(a, grid, 32 * warps, s);
  else e4m3 ? append<false, MOE_DT_E4M3>(a, grid, 32 * warps, s) : append<false, MOE_DT_INT8>(a, grid, 32 * warps, s);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_q8(const KvReadQ8Args& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  note_launch();
  if (a.kv.dtype == MOE_DT_E4M3) read_as<MOE_DT_E4M3>(a, s);
  else read_as<MOE_DT_INT8>(a, s);
  return cudaGetLastError();
}

}  // namespace moe
