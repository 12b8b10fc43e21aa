// Appending a chunk's keys and values to a paged cache.
//
// What bounds it: memory, and for a decode step latency.  Each new element is
// read once and written once.  One warp per token: it finds the token's
// sequence with a 32-way search of cu_q (two rounds for up to 1024
// sequences), forms the page address once, and copies the token's heads in
// 16-byte vectors; several vectors per lane are in flight before the first
// store.  5257 tokens of 8 heads of 128 (43 MB): 8.7 us, 4.9 TB/s with the
// launch; 64 tokens: 2.8 us.
#include "moe_kv.cuh"

namespace moe {
namespace {

template <typename V>
__global__ void __launch_bounds__(128) kv_append_kernel(const KvAppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  // the first vectors are asked for before the token's page is looked up
  constexpr int kPer = sizeof(V) / 2, kBatch = 4;
  const int vecs = a.kv.D / kPer, total = a.kv.Hkv * vecs;
  const uint16_t* k = static_cast<const uint16_t*>(a.k) + (int64_t)t * a.k_stride;
  const uint16_t* v = static_cast<const uint16_t*>(a.v) + (int64_t)t * a.v_stride;
  V kb[kBatch], vb[kBatch];
  const auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + 32 * u;
      if (i < total) {
        const int h = i / vecs, c = (i - h * vecs) * kPer;
        kb[u] = *reinterpret_cast<const V*>(k + h * a.k_head_stride + c);
        vb[u] = *reinterpret_cast<const V*>(v + h * a.v_head_stride + c);
      }
    }
  };
  load(lane);
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
  uint16_t* kc = static_cast<uint16_t*>(a.k_cache) + (int64_t)page * a.kv.k_page_stride + slot * a.kv.k_row_stride;
  uint16_t* vc = static_cast<uint16_t*>(a.v_cache) + (int64_t)page * a.kv.v_page_stride + slot * a.kv.v_row_stride;
  for (int i0 = lane; i0 < total; i0 += 32 * kBatch) {
    if (i0 != lane) load(i0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + 32 * u;
      if (i < total) {
        const int h = i / vecs, c = (i - h * vecs) * kPer;
        *reinterpret_cast<V*>(kc + h * a.kv.k_head_stride + c) = kb[u];
        *reinterpret_cast<V*>(vc + h * a.kv.v_head_stride + c) = vb[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int warps = a.T <= 4 * num_sms() ? 1 : 4;
  const unsigned grid = (unsigned)((a.T + warps - 1) / warps);
  note_launch();
  if (a.wide) kv_append_kernel<uint4><<<grid, 32 * warps, 0, s>>>(a);
  else kv_append_kernel<uint16_t><<<grid, 32 * warps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
