// Routing of given logits: softmax or sigmoid scores, a bias that only takes
// part in the selection, expert groups, top-k and renormalised gates.
//
// One warp per token; the logits are read once and stay in registers.
//
// The selection is the one that 64-bit keys give.  Keys are formed in fp32
// with a bound on their error; lane s re-derives the key of the s-th choice
// and compares it with the next one.  Where a gap (between neighbours of the
// result, or between the last kept and the first dropped group) is within the
// two bounds, fp32 cannot tell, and the warp decides that token again with
// fp64 keys.  Without a bias the order of the keys is that of the logits,
// which are compared exactly.  A gap of exactly equal inputs (same logit, same
// bias) is a tie in any precision and goes to the lower index.
//
// Error bound of a key p + b, in units of 2^-24: expf is within 2 ulp, so the
// sigmoid (one addition, one division) is within 6 p; the softmax adds the
// rounding of l - m (|l - m| p, below 104 p for any p that fp32 can hold) and
// the sum's (one rounding per element of a lane and per shuffle).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr float kUlp = 5.9604645e-08f;  // 2^-24
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t at) {
  float v;
  if (a.dtype == MOE_DT_F32) v = static_cast<const float*>(a.logits)[at];
  else if (a.dtype == MOE_DT_BF16) v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at]);
  else v = __half2float(static_cast<const __half*>(a.logits)[at]);
  return v != v ? -INFINITY : v;
}

__device__ __forceinline__ uint32_t order_key(float v) {  // as logit_key; never 0, which marks a taken entry
  return logit_key(v);
}

// softmax statistics of a token; sigmoid uses neither
struct Stats {
  float m, sum;
};

__device__ __forceinline__ float score32(float l, int route, Stats st) {
  if (route == MOE_ROUTE_SIGMOID) return 1.0f / (1.0f + expf(-l));
  if (st.m == -INFINITY) return 0.0f;
  return (l == st.m ? 1.0f : expf(l - st.m)) / st.sum;
}

__device__ __forceinline__ double score64(float l, int route, float m, double sum) {
  if (route == MOE_ROUTE_SIGMOID) return 1.0 / (1.0 + exp(-(double)l));
  if (m == -INFINITY) return 0.0;
  return (l == m ? 1.0 : exp((double)l - (double)m)) / sum;
}

__device__ __forceinline__ double shfl_xor_d(double v, int o) { return __shfl_xor_sync(kAll, v, o); }

// The token decided with fp64 keys: rare, so written for size.  Lane r returns
// the r-th choice.  Keys are recomputed from the logits in
// global memory, one element at a time.
__device__ __noinline__ int select64(const RouteArgs& a, int64_t row, int lane, float m) {
  const int npl = (a.E + 31) / 32, e0 = lane * npl;
  double sum = 0.0;
  if (a.route == MOE_ROUTE_SOFTMAX && m != -INFINITY) {
    for (int j = 0; j < npl; ++j)
      if (e0 + j < a.E) {
        const float l = load_logit(a, row + e0 + j);
        sum += l == m ? 1.0 : exp((double)l - (double)m);
      }
    for (int o = 16; o > 0; o >>= 1) sum += shfl_xor_d(sum, o);
  }
  const int gs = a.E / a.n_group;
  uint32_t kept = kAll;  // bit g: group g may be used
  if (a.n_group > 1) {
    // lane g scores group g
    double score = -INFINITY;
    if (lane < a.n_group) {
      double first = -INFINITY, second = -INFINITY;
      for (int e = lane * gs; e < lane * gs + gs; ++e) {
        const double key = score64(load_logit(a, row + e), a.route, m, sum) + (a.bias ? (double)a.bias[e] : 0.0);
        if (key > first) second = first, first = key;
        else if (key > second) second = key;
      }
      score = a.group_score == MOE_GROUP_TOP2 && gs > 1 ? first + second : first;
    }
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
      const double other = __shfl_sync(kAll, score, g);
      rank += other > score || (other == score && g < lane);
    }
    kept = __ballot_sync(kAll, lane < a.n_group && rank < a.topk_group);
  }
  uint32_t used = 0;  // bit j: the lane's element j was chosen
  int mine = 0;
  for (int r = 0; r < a.k; ++r) {
    double best = -INFINITY;
    int at = INT_MAX;
    for (int j = 0; j < npl; ++j) {
      const int e = e0 + j;
      if (e >= a.E || (used >> j & 1) || !(kept >> (e / gs) & 1)) continue;
      const float l = load_logit(a, row + e);
      const double key = a.bias ? score64(l, a.route, m, sum) + (double)a.bias[e] : (double)l;
      if (at == INT_MAX || key > best) best = key, at = e;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = shfl_xor_d(best, o);
      const int oa = __shfl_xor_sync(kAll, at, o);
      if (oa != INT_MAX && (at == INT_MAX || ob > best || (ob == best && oa < at))) best = ob, at = oa;
    }
    if (at / npl == lane) used |= 1u << (at - e0);
    if (lane == r) mine = at;
  }
  return mine;
}

// NP >= ceil(E / 32): elements per lane
template <int NP>
__global__ void __launch_bounds__(128) route_grouped_kernel(const RouteArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int64_t row = (int64_t)t * a.stride;
  const int npl = (a.E + 31) / 32, e0 = lane * npl;
  float l[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) l[j] = j < npl && e0 + j < a.E ? load_logit(a, row + e0 + j) : -INFINITY;

  Stats st{0.0f, 1.0f};
  if (a.route == MOE_ROUTE_SOFTMAX) {
    float m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NP; ++j) m = fmaxf(m, l[j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    if (m != -INFINITY) {
#pragma unroll
      for (int j = 0; j < NP; ++j) sum += l[j] == m ? 1.0f : expf(l[j] - m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    st = Stats{m, sum};
  }
  const float bound = a.route == MOE_ROUTE_SIGMOID ? 6.0f : (float)(npl + 130);

  // ordering keys: p + b with a bias, the logits themselves without
  uint32_t key[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const bool in = j < npl && e0 + j < a.E;
    const float v = in && a.bias ? score32(l[j], a.route, st) + a.bias[e0 + j] : l[j];
    key[j] = in ? order_key(v) : 0u;
  }

  bool unsure = false;
  if (a.n_group > 1) {
    const int gs = a.E / a.n_group;
    // the two largest keys of each group, lane g keeping group g's
    float my_score = -INFINITY, my_err = 0.0f;
    for (int g = 0; g < a.n_group; ++g) {
      float first = -INFINITY, second = -INFINITY;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int e = e0 + j;
        if (j < npl && e < a.E && e / gs == g) {
          const float v = a.bias ? key_logit(key[j]) : a.group_score == MOE_GROUP_TOP2 ? score32(l[j], a.route, st) : l[j];
          if (v > first) second = first, first = v;
          else if (v > second) second = v;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float f = __shfl_xor_sync(kAll, first, o), s2 = __shfl_xor_sync(kAll, second, o);
        second = fmaxf(fminf(first, f), fmaxf(second, s2));
        first = fmaxf(first, f);
      }
      if (lane == g) {
        const bool two = a.group_score == MOE_GROUP_TOP2 && gs > 1;
        my_score = two ? first + second : first;
        // each key within (bound * p + |key|) ulp, p <= 1; without a bias a single logit is exact
        my_err = a.bias || two ? kUlp * (fabsf(my_score) + fabsf(first) + fabsf(second == -INFINITY ? 0.0f : second) +
                                         (two ? 2.0f : 1.0f) * bound)
                               : 0.0f;
      }
    }
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
      const float other = __shfl_sync(kAll, my_score, g);
      rank += other > my_score || (other == my_score && g < lane);
    }
    const bool in = lane < a.n_group && rank < a.topk_group;
    const uint32_t kept = __ballot_sync(kAll, in);
    // the last kept against the first dropped group
    if (a.topk_group < a.n_group) {
      const unsigned last = __ballot_sync(kAll, lane < a.n_group && rank == a.topk_group - 1);
      const unsigned next = __ballot_sync(kAll, lane < a.n_group && rank == a.topk_group);
      const float s0 = __shfl_sync(kAll, my_score, __ffs(last) - 1), s1 = __shfl_sync(kAll, my_score, __ffs(next) - 1);
      const float x0 = __shfl_sync(kAll, my_err, __ffs(last) - 1), x1 = __shfl_sync(kAll, my_err, __ffs(next) - 1);
      unsure = x0 + x1 > 0.0f && s0 - s1 <= x0 + x1;
    }
#pragma unroll
    for (int j = 0; j < NP; ++j)
      if (key[j] && !(kept >> ((e0 + j) / gs) & 1)) key[j] = 0u;
  }

  // the k largest, and with a bias the one after them
  const int avail = a.n_group > 1 ? a.topk_group * (a.E / a.n_group) : a.E;
  const int rounds = a.bias && a.k < avail ? a.k + 1 : a.k;
  int mine = 0;
  for (int r = 0; r < rounds; ++r) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < NP; ++j) best = max(best, key[j]);
    const uint32_t top = __reduce_max_sync(kAll, best);
    const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
    int at = 0;
    if (lane == owner) {
      bool done = false;
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (!done && key[j] == top) done = true, key[j] = 0u, at = e0 + j;
    }
    at = __shfl_sync(kAll, at, owner);
    if (lane == r) mine = at;
  }

  float lg = 0.0f;
  if (lane < rounds) lg = load_logit(a, row + mine);
  if (a.bias) {
    const float b = lane < rounds ? a.bias[mine] : 0.0f;
    const float p = score32(lg, a.route, st), v = p + b;
    const float err = kUlp * (bound * p + fabsf(v));
    const float v1 = __shfl_down_sync(kAll, v, 1), err1 = __shfl_down_sync(kAll, err, 1);
    const float l1 = __shfl_down_sync(kAll, lg, 1), b1 = __shfl_down_sync(kAll, b, 1);
    const bool same = lg == l1 && b == b1;
    unsure |= __any_sync(kAll, lane + 1 < rounds && !same && v - v1 <= err + err1);
  }
  if (unsure) {
    mine = select64(a, row, lane, st.m);
    if (lane < a.k) lg = load_logit(a, row + mine);
  }

  const float p = lane < a.k ? score32(lg, a.route, st) : 0.0f;
  float g = p;
  if (a.renorm) {
    float sum = p;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    g = sum > 0.0f ? p / sum : 0.0f;
  }
  if (lane < a.k) {
    a.ids[(int64_t)t * a.k + lane] = mine;
    a.gates[(int64_t)t * a.k + lane] = g * a.scale;
  }
}

}  // namespace

cudaError_t launch_route_grouped(const RouteArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int npl = (a.E + 31) / 32;
  const int warps = a.T <= 4 * num_sms() ? 1 : 4;  // few tokens: one CTA each
  const unsigned grid = (unsigned)((a.T + warps - 1) / warps);
  note_launch();
  if (npl <= 2) route_grouped_kernel<2><<<grid, 32 * warps, 0, s>>>(a);
  else if (npl <= 4) route_grouped_kernel<4><<<grid, 32 * warps, 0, s>>>(a);
  else if (npl <= 8) route_grouped_kernel<8><<<grid, 32 * warps, 0, s>>>(a);
  else if (npl <= 16) route_grouped_kernel<16><<<grid, 32 * warps, 0, s>>>(a);
  else route_grouped_kernel<32><<<grid, 32 * warps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
