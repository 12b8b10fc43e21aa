// The paged key/value cache: what the kernels that write and read it share.
#pragma once

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

// Rows and keys of sequence b, checked against the call's sizes: every index
// that a kernel forms from them is in range.
__device__ __forceinline__ SeqInfo seq_info(const moe_kv_desc& kv, const int32_t* cu_q, const int32_t* kv_len, int T,
                                            int b) {
  const int q0 = __ldg(cu_q + b), q1 = __ldg(cu_q + b + 1), len = __ldg(kv_len + b);
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= T && len >= 0 && len <= (int64_t)kv.max_pages * kv.page_size;
  return ok ? SeqInfo{q0, q1 - q0, len, true} : SeqInfo{0, 0, 0, false};
}

// The first key that a row which may see the keys below `hi` does see.  hi is
// at or below 0 for a row before the first key; the window is any int, so it
// is not taken off a negative number.
__device__ __forceinline__ int window_lo(int hi, int window) { return window > 0 ? max(max(hi, 0) - window, 0) : 0; }

// the last b with cu_q[b] <= t (cu_q ascending); the whole warp takes part
__device__ __forceinline__ int find_seq(const int32_t* cu_q, int n_seqs, int t, int lane) {
  int lo = 0, n = n_seqs;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && (at == 0 || __ldg(cu_q + lo + at) <= t);
    const unsigned mask = __ballot_sync(0xffffffffu, le);
    const int last = 31 - __clz((int)mask);
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

}  // namespace moe
