// Attention over an 8-bit paged cache, the general kernel: any head size that
// is a multiple of 8 up to 256, any page size, codes on 8-byte boundaries.  One
// CTA per (token, query head); its four warps take every fourth key each, with
// the running maximum and sum of an online softmax, and their results are
// joined in shared memory.  It reads each key once per query head, so it is the
// form for sizes that the tensor-core kernel does not take, not for speed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_kv.cuh"
#include "moe_q8.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

template <typename T, int FMT>
__global__ void __launch_bounds__(32 * kWarps) attn_q8_general_kernel(const AttnQ8Args g) {
  const AttnArgs& a = g.a;
  __shared__ float s_m[kWarps], s_l[kWarps];
  __shared__ float s_o[kWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = blockIdx.y, kvh = head / (a.Hq / a.kv.Hkv);
  const int D = a.kv.D;
  const bool act = lane * 8 < D;
  if (blockIdx.x == 0 && blockIdx.y == 0)  // sequences without tokens of this call are looked at too
    for (int b = threadIdx.x; b < a.kv.n_seqs; b += blockDim.x)
      if (!seq_info(a.kv, a.cu_q, a.kv_len, a.T, b).ok) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int b = find_seq(a.cu_q, a.kv.n_seqs, t, lane);
    const SeqInfo s = seq_info(a.kv, a.cu_q, a.kv_len, a.T, b);
    if (!s.ok || t < s.q0 || t >= s.q0 + s.n) continue;  // uniform over the CTA
    const int pos = s.kv - s.n + (t - s.q0);
    const int hi = pos + 1, lo = window_lo(hi, a.window);
    float q[8] = {};
    if (act) {
      const T* p = static_cast<const T*>(a.q) + (int64_t)t * a.q_stride + head * a.q_head_stride + lane * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = (float)p[i];
    }
    float m = -INFINITY, l = 0.0f, o[8] = {};
    for (int j = lo + warp; j < hi; j += kWarps) {
      const int page = __ldg(a.table + (int64_t)b * a.kv.table_stride + j / a.kv.page_size);
      const bool in = page >= 0 && page < a.kv.num_pages;
      if (!in && lane == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      const int64_t slot = j % a.kv.page_size;
      float dot = 0.0f, e = 0.0f, v[8] = {};
      if (in) {
        if (act) {
          float k[8];
          const uint2 kw = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.k_cache) + page * a.kv.k_page_stride +
                                                           slot * a.kv.k_row_stride + kvh * a.kv.k_head_stride + lane * 8);
          const uint2 vw = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.v_cache) + page * a.kv.v_page_stride +
                                                           slot * a.kv.v_row_stride + kvh * a.kv.v_head_stride + lane * 8);
          four_values<FMT>(kw.x, k);
          four_values<FMT>(kw.y, k + 4);
          four_values<FMT>(vw.x, v);
          four_values<FMT>(vw.y, v + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fmaf(q[i], k[i], dot);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
        dot *= a.scale * g.sc.k[page * g.sc.k_page_stride + slot * g.sc.k_row_stride + kvh * g.sc.k_head_stride];
        e = g.sc.v[page * g.sc.v_page_stride + slot * g.sc.v_row_stride + kvh * g.sc.v_head_stride];
      }
      const float m1 = fmaxf(m, dot);
      const float f = m1 == -INFINITY ? 1.0f : expf(m - m1);
      const float p = m1 == -INFINITY ? (dot == m1 ? 0.0f : dot) : expf(dot - m1);  // (a maximum skips NaN, the sum does not)
      m = m1;
      l = l * f + p;
      const float pe = p * e;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(pe, v[i], o[i] * f);
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
    if (mm == -INFINITY)  // every score -inf or not a number: the sums tell which
      for (int w = 0; w < kWarps; ++w) ll += s_l[w];
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

cudaError_t launch_attn_q8_general(const AttnQ8Args& g, cudaStream_t s) {
  if (g.a.T == 0) return cudaSuccess;
  const dim3 grid((unsigned)(g.a.T < 65536 ? g.a.T : 65536), (unsigned)g.a.Hq);
  note_launch();
  const bool e4m3 = g.a.kv.dtype == MOE_DT_E4M3;
  if (g.x_dtype == MOE_DT_BF16)
    e4m3 ? attn_q8_general_kernel<__nv_bfloat16, MOE_DT_E4M3><<<grid, 32 * kWarps, 0, s>>>(g)
         : attn_q8_general_kernel<__nv_bfloat16, MOE_DT_INT8><<<grid, 32 * kWarps, 0, s>>>(g);
  else
    e4m3 ? attn_q8_general_kernel<__half, MOE_DT_E4M3><<<grid, 32 * kWarps, 0, s>>>(g)
         : attn_q8_general_kernel<__half, MOE_DT_INT8><<<grid, 32 * kWarps, 0, s>>>(g);
  return cudaGetLastError();
}

}  // namespace moe
