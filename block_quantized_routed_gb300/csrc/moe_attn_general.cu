// Attention over a paged cache, the general kernel: any head size that is a
// multiple of 8 up to 256 and any page size.  One CTA per (token, query head);
// its four warps take every fourth key each, with the running maximum and sum
// of an online softmax, and their results are joined in shared memory.  It
// reads each key once per query head, so it is the form for sizes that the
// tensor-core kernel does not take, not for speed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_kv.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& raw, float* v) {
  T e[8];
  *reinterpret_cast<uint4*>(e) = raw;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2) v[i] = (float)e[i];
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) attn_general_kernel(const AttnArgs a) {
  __shared__ float s_m[kWarps], s_l[kWarps];
  __shared__ float s_o[kWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = blockIdx.y, kvh = head / (a.Hq / a.kv.Hkv);
  const int D = a.kv.D;
  const bool act = lane * 8 < D;
  // the token's sequence: a linear walk, as this kernel is not the fast one
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    SeqInfo s{0, 0, 0, true};
    int b = 0;
    for (; b < a.kv.n_seqs; ++b) {
      s = seq_info(a.kv, a.cu_q, a.kv_len, a.T, b);
      if (!s.ok && threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      if (s.ok && t >= s.q0 && t < s.q0 + s.n) break;
    }
    if (b == a.kv.n_seqs) continue;  // uniform over the CTA
    const int pos = s.kv - s.n + (t - s.q0);
    const int hi = pos + 1, lo = window_lo(hi, a.window);
    float q[8];
    if (act) {
      unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (int64_t)t * a.q_stride +
                                                 head * a.q_head_stride + lane * 8), q);
    }
    float m = -INFINITY, l = 0.0f, o[8] = {};
    for (int j = lo + warp; j < hi; j += kWarps) {
      const int page = __ldg(a.table + (int64_t)b * a.kv.table_stride + j / a.kv.page_size);
      const bool in = page >= 0 && page < a.kv.num_pages;
      if (!in && lane == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      const int64_t slot = j % a.kv.page_size;
      float kv[8] = {}, dot = 0.0f;
      if (act && in) {
        unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_cache) + page * a.kv.k_page_stride +
                                                   slot * a.kv.k_row_stride + kvh * a.kv.k_head_stride + lane * 8), kv);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(q[i], kv[i], dot);
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
      dot *= a.scale;
      const float m1 = fmaxf(m, dot);
      const float f = m1 == -INFINITY ? 1.0f : expf(m - m1);
      const float p = m1 == -INFINITY ? (dot == m1 ? 0.0f : dot) : expf(dot - m1);  // (a maximum skips NaN, the sum does not)
      m = m1;
      l = l * f + p;
      float v[8] = {};
      if (act && in)
        unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.v_cache) + page * a.kv.v_page_stride +
                                                   slot * a.kv.v_row_stride + kvh * a.kv.v_head_stride + lane * 8), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(p, v[i], o[i] * f);
    }
    __syncthreads();  // the previous token's join has been read
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    if (act) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s_o[warp][lane * 8 + i] = o[i];
    }
    __syncthreads();
    float mm = -INFINITY, ll = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
    float f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[w] = mm == -INFINITY ? 0.0f : expf(s_m[w] - mm);
      ll += f[w] * s_l[w];
    }
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v = fmaf(f[w], s_o[w][c], v);
      static_cast<T*>(a.out)[(int64_t)t * a.o_stride + head * a.o_head_stride + c] = (T)(ll == 0.0f ? 0.0f : v / ll);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)t * a.Hq + head] = ll == 0.0f ? -INFINITY : mm + logf(ll);
  }
}

}  // namespace

cudaError_t launch_attn_general(const AttnArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const dim3 grid((unsigned)(a.T < 65536 ? a.T : 65536), (unsigned)a.Hq);
  note_launch();
  if (a.kv.dtype == MOE_DT_BF16) attn_general_kernel<__nv_bfloat16><<<grid, 32 * kWarps, 0, s>>>(a);
  else attn_general_kernel<__half><<<grid, 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
