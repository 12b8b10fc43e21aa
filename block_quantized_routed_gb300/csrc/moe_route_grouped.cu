// Routing of given logits: softmax or sigmoid scores, a bias that only takes
// part in the selection, expert groups, top-k and renormalised gates.
//
// One warp per token; the logits are read once and stay in registers.
//
// The selection is the one that 64-bit keys give.  Keys are formed in fp32
// with a bound on their error; lane s re-derives the key of the s-th choice
// and compares it with the next one, the k-th with the first that is not its
// equal, by a bound that holds for all that was not chosen.  Where a gap
// (between neighbours of the result, below the k-th, or between any kept and
// any dropped group) is within the two bounds, fp32 cannot tell: the
// choices in question, and those that might displace the last of them, are
// ranked again by fp64 keys, and likewise the elements that make up the
// groups' scores, one key per lane.  (Deciding such a
// token with fp64 keys of all its experts takes a warp tens of microseconds on
// this part's few fp64 units: it is left for more than 32 such elements.)
// Without a bias the order of the keys is that of the logits, which are
// compared exactly.  A gap of exactly equal inputs (same logit, same bias) is a
// tie in any precision and goes to the lower index.
//
// What bounds it: the chain of dependent warp-wide steps of the rounds (largest
// head, its owner, the shift of the owner's keys), about 900 warp instructions
// a token at 256 experts and k = 8, with 9 of an SM's 13.5 CTAs resident (8192
// tokens: 14.9 us in 8 groups with a bias, of which issue takes 6; their 8 MB
// take 1.3); for few tokens the latency of the rounds, and more so of code that
// is fetched for the first time.  So a lane holds no more keys than it has to
// (528 experts in lanes of 20 and not 32, one warp per CTA: 12 to 7.5 us).
//
// Error bound of a key p + b, in units of 2^-24.  exp32 is within 4 (2 ulp) and
// 1.5 |x| (its argument is scaled and rounded).  Sigmoid: the error of e^-l
// reaches p times 1 - p, and p (1 - p) |l| < 0.3, so with the addition and the
// reciprocal 8 p + 1 covers it.  Softmax, x = l - m: p 1.5 |x| < 0.6 for the
// element itself; in the sum the errors' weighted mean is 1.5 (ln E + 1) < 12,
// and each addition in a lane and each shuffle rounds: (npl + 32) p + 1 covers it.
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

// as logit_key, for a v that is no NaN: larger v, larger key; never 0, which marks a taken entry
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and +0 are the same logit
  return max(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), 1u);  // (a NaN bias: some key, never 0)
}

// softmax statistics of a token; sigmoid uses neither
struct Stats {
  float m, inv_sum;
};

__device__ __forceinline__ float exp32(float x) {  // 2 ulp, and the rounding of the argument: |x| ulp
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504088896341f));
  return y;
}
__device__ __forceinline__ float rcp32(float x) {  // 1 ulp; 0 at infinity
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// sigmoid: m and inv_sum unused; softmax: the row's maximum and the reciprocal of its sum
__device__ __forceinline__ float score32(float l, int route, Stats st) {
  if (route == MOE_ROUTE_SIGMOID) return rcp32(1.0f + exp32(-l));
  if (st.m == -INFINITY) return 0.0f;
  return (l == st.m ? 1.0f : exp32(l - st.m)) * st.inv_sum;
}

// An infinite key comes from an infinite bias and is exact.
__device__ __forceinline__ float magnitude(float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.0f; }
// v certainly comes before v1 (which it was not after in fp32)
__device__ __forceinline__ bool above(float v, float v1, float tol) {
  return v - v1 > tol || (v == v1 && fabsf(v) == INFINITY);
}

__device__ __forceinline__ double score64(float l, int route, float m, double sum) {
  if (route == MOE_ROUTE_SIGMOID) return 1.0 / (1.0 + exp(-(double)l));
  if (m == -INFINITY) return 0.0;
  return (l == m ? 1.0 : exp((double)l - (double)m)) / sum;
}

__device__ __forceinline__ double shfl_xor_d(double v, int o) { return __shfl_xor_sync(kAll, v, o); }

// the softmax's denominator in fp64 (1 for the sigmoid)
__device__ __noinline__ double sum64(const RouteArgs& a, int64_t row, int lane, float m) {
  if (a.route != MOE_ROUTE_SOFTMAX || m == -INFINITY) return 1.0;
  double sum = 0.0;
  for (int e = lane; e < a.E; e += 32) {
    const float l = load_logit(a, row + e);
    sum += l == m ? 1.0 : exp((double)l - (double)m);
  }
  for (int o = 16; o > 0; o >>= 1) sum += shfl_xor_d(sum, o);
  return sum;
}

// The token decided with fp64 keys throughout (its groups, or more than 32
// candidates, are too near to one another): lane r returns the r-th choice.
// buf: E doubles of the warp's shared memory.
__device__ __noinline__ int select64(const RouteArgs& a, int64_t row, int lane, float m, double* buf) {
  const double sum = sum64(a, row, lane, m);
  const int gs = a.E / a.n_group;
  __syncwarp();
  for (int e = lane; e < a.E; e += 32)
    buf[e] = score64(load_logit(a, row + e), a.route, m, sum) + (a.bias ? (double)a.bias[e] : 0.0);
  __syncwarp();
  uint32_t kept = kAll;  // bit g: group g may be used
  if (a.n_group > 1) {
    double score = -INFINITY;  // lane g scores group g
    if (lane < a.n_group) {
      double first = -INFINITY, second = -INFINITY;
      for (int j = 0; j < gs; ++j) {
        const double key = buf[lane * gs + j];
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
  uint32_t used = 0;  // bit j: element lane + 32 j was chosen
  int mine = 0;
  for (int r = 0; r < a.k; ++r) {
    double best = -INFINITY;
    int at = INT_MAX;
    for (int j = 0, e = lane; e < a.E; ++j, e += 32) {
      if ((used >> j & 1) || !(kept >> (e / gs) & 1)) continue;
      const double key = a.bias ? buf[e] : (double)load_logit(a, row + e);
      if (at == INT_MAX || key > best) best = key, at = e;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = shfl_xor_d(best, o);
      const int oa = __shfl_xor_sync(kAll, at, o);
      if (oa != INT_MAX && (at == INT_MAX || ob > best || (ob == best && oa < at))) best = ob, at = oa;
    }
    if ((at & 31) == lane) used |= 1u << (at >> 5);
    if (lane == r) mine = at;
  }
  return mine;
}

// The choices among n <= 32 candidates, lane i holding candidate e (logit l),
// by fp64 keys: one key per lane.  Lane r returns the r-th choice.
__device__ __noinline__ int rank64(const RouteArgs& a, int64_t row, int lane, float m, int n, int e, float l) {
  const double sum = sum64(a, row, lane, m);
  double key = -INFINITY;
  if (lane < n) key = score64(l, a.route, m, sum) + (double)a.bias[e];
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const double other = __shfl_sync(kAll, key, i);
    const int oe = __shfl_sync(kAll, e, i);
    rank += other > key || (other == key && oe < e);
  }
  if (lane >= n) rank = 64;
  int mine = 0;
  for (int i = 0; i < n; ++i) {
    const int ri = __shfl_sync(kAll, rank, i), oe = __shfl_sync(kAll, e, i);
    if (ri == lane) mine = oe;
  }
  return mine;
}

// The groups' scores by fp64 keys of the n <= 32 elements `list` that may be
// among a group's two largest, one per lane: bit g of the result is set for
// the topk_group best groups.
__device__ __noinline__ uint32_t groups64(const RouteArgs& a, int64_t row, int lane, float m, int n, const int* list) {
  const double sum = sum64(a, row, lane, m);
  const int e = lane < n ? list[lane] : 0, gs = a.E / a.n_group;
  double key = -INFINITY;
  if (lane < n) key = score64(load_logit(a, row + e), a.route, m, sum) + (a.bias ? (double)a.bias[e] : 0.0);
  double first = -INFINITY, second = -INFINITY;  // lane g: of group g
  for (int i = 0; i < n; ++i) {
    const double k = __shfl_sync(kAll, key, i);
    const int g = __shfl_sync(kAll, e, i) / gs;
    if (g != lane) continue;
    if (k > first) second = first, first = k;
    else if (k > second) second = k;
  }
  const double score = lane >= a.n_group ? -INFINITY
                       : a.group_score == MOE_GROUP_TOP2 && gs > 1 ? first + second : first;
  int rank = 0;
  for (int g = 0; g < a.n_group; ++g) {
    const double other = __shfl_sync(kAll, score, g);
    rank += other > score || (other == score && g < lane);
  }
  return __ballot_sync(kAll, lane < a.n_group && rank < a.topk_group);
}

// The gate of lane r's choice (logit l, r < k), before the scale.  Renormalised gates are ratios of scores, formed with
// the largest exponential of the choices divided out, so that they hold where the scores themselves are below fp32's
// range, and so that the approximate exponential sees small arguments: sigmoid(l) = e^min(l, 0) / (1 + e^-|l|),
// softmax e^l / sum.
__device__ __forceinline__ float gate(const RouteArgs& a, int lane, float l, Stats st) {
  const bool chosen = lane < a.k, sigmoid = a.route == MOE_ROUTE_SIGMOID;
  const float x = sigmoid ? fminf(l, 0.0f) : l;
  float top = a.renorm ? chosen ? x : -INFINITY : sigmoid ? 0.0f : st.m;
  if (a.renorm) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  }
  float w = !chosen || x == -INFINITY ? 0.0f : x == top ? 1.0f : exp32(x - top);
  if (sigmoid) w *= rcp32(1.0f + exp32(-fabsf(l)));
  if (!a.renorm) return sigmoid ? w : w > 0.0f ? w * st.inv_sum : 0.0f;  // (a row of -inf: no sum)
  float sum = w;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  return sum > 0.0f ? w / sum : 0.0f;
}

// The largest key at or below key_k of an element that is not the equal of e_k (another logit or bias); -inf: none.
// s_key: [element of a lane][lane] keys.
__device__ __noinline__ float next_other(const RouteArgs& a, int64_t row, int e_k, uint32_t key_k, const uint32_t* s_key) {
  const int lane = threadIdx.x & 31, npl = (a.E + 31) / 32, e0 = lane * npl;
  const float l = load_logit(a, row + e_k), b = __ldg(a.bias + e_k);
  uint32_t top = 0;
  for (int j = 0; j < npl && e0 + j < a.E; ++j) {
    const uint32_t key = s_key[j * 32 + lane];
    if (key > top && key <= key_k && !(load_logit(a, row + e0 + j) == l && __ldg(a.bias + e0 + j) == b)) top = key;
  }
  top = __reduce_max_sync(kAll, top);
  return top ? key_logit(top) : -INFINITY;
}

// the two largest of two pairs, each in order
__device__ __forceinline__ void top2_join(float& first, float& second, float f, float s) {
  second = fmaxf(fminf(first, f), fmaxf(second, s));
  first = fmaxf(first, f);
}

__device__ __forceinline__ void top2_add(float& first, float& second, float v) {
  second = fmaxf(second, fminf(first, v));
  first = fmaxf(first, v);
}

// Batcher's odd-even merge sort of N keys, largest first: that of the next
// power of two without the comparisons that reach past N (where the smallest
// keys would lie and stay).
// (P, Q: the step, as template arguments so that every index is a constant.)
template <int N, int P, int Q>
__device__ __forceinline__ void sort_step(uint32_t (&k)[N]) {
#pragma unroll
  for (int j = Q % P; j + Q < N; j += 2 * Q)
#pragma unroll
    for (int i = 0; i < Q; ++i)
      if (i + j + Q < N && (i + j) / (2 * P) == (i + j + Q) / (2 * P)) {
        const uint32_t x = k[i + j], y = k[i + j + Q];
        k[i + j] = max(x, y);
        k[i + j + Q] = min(x, y);
      }
  if constexpr (Q > 1) sort_step<N, P, Q / 2>(k);
  else if constexpr (2 * P < N) sort_step<N, 2 * P, 2 * P>(k);
}

// NP >= ceil(E / 32): elements per lane; lane i holds elements i * npl on.
// VEC: npl = NP, E = 32 * NP, and the rows and the bias are 16-byte aligned (wide loads).
template <int NP, bool VEC>
__global__ void __launch_bounds__(128) route_grouped_kernel(const RouteArgs a) {
  __shared__ double s_buf[4][NP * 32];  // keys: of groups that do not fall on lane boundaries (fp32); of select64
  __shared__ int s_list[4][32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int t = blockIdx.x * (blockDim.x >> 5) + wid;
  if (t >= a.T) return;
  const int64_t row = (int64_t)t * a.stride;
  const int npl = VEC ? NP : (a.E + 31) / 32, e0 = lane * npl;
  const int have = VEC ? NP : max(0, min(npl, a.E - e0));  // elements of this lane
  float l[NP];
  if constexpr (VEC) {
    if (a.dtype == MOE_DT_F32) {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + row + e0);
#pragma unroll
      for (int j = 0; j < NP / 4; ++j) {
        const float4 v = __ldg(src + j);
        l[4 * j] = v.x, l[4 * j + 1] = v.y, l[4 * j + 2] = v.z, l[4 * j + 3] = v.w;
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.logits) + row + e0);
#pragma unroll
      for (int j = 0; j < NP / 8; ++j) {
        const uint4 v = __ldg(src + j);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 f;
          if (a.dtype == MOE_DT_BF16) f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
          else f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          l[8 * j + 2 * i] = f.x, l[8 * j + 2 * i + 1] = f.y;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) l[j] = l[j] != l[j] ? -INFINITY : l[j];
  } else {  // (the type is looked at once, so that the loads are under way together)
    const auto load = [&](auto* src, auto wide) {
#pragma unroll
      for (int j = 0; j < NP; ++j) l[j] = j < have ? wide(src[row + e0 + j]) : -INFINITY;
    };
    if (a.dtype == MOE_DT_F32) load(static_cast<const float*>(a.logits), [](float v) { return v; });
    else if (a.dtype == MOE_DT_BF16)
      load(static_cast<const __nv_bfloat16*>(a.logits), [](__nv_bfloat16 v) { return __bfloat162float(v); });
    else load(static_cast<const __half*>(a.logits), [](__half v) { return __half2float(v); });
#pragma unroll
    for (int j = 0; j < NP; ++j) l[j] = l[j] != l[j] ? -INFINITY : l[j];
  }

  float b[NP];  // the bias
  if (a.bias) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < NP; j += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(a.bias + e0 + j));
        b[j] = v.x, b[j + 1] = v.y, b[j + 2] = v.z, b[j + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) b[j] = j < have ? __ldg(a.bias + e0 + j) : 0.0f;
    }
  }

  Stats st{0.0f, 1.0f};  // of the softmax
  if (a.route == MOE_ROUTE_SOFTMAX) {
    float m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NP; ++j) m = fmaxf(m, l[j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    if (m != -INFINITY) {
#pragma unroll
      for (int j = 0; j < NP; ++j) sum += l[j] == m ? 1.0f : exp32(l[j] - m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    st = Stats{m, 1.0f / sum};
  }
  const float bound = a.route == MOE_ROUTE_SIGMOID ? 8.0f : (float)(npl + 32);

  // ordering keys: p + b with a bias, the logits themselves without; a group's
  // score takes p (+ b) where it adds two keys
  const bool scored = a.bias != nullptr;
  uint32_t key[NP];
  if (scored) {
#pragma unroll
    for (int j = 0; j < NP; ++j) key[j] = j < have ? order_key(score32(l[j], a.route, st) + b[j]) : 0u;
  } else {
#pragma unroll
    for (int j = 0; j < NP; ++j) key[j] = j < have ? order_key(l[j]) : 0u;
  }

  bool unsure = false;
  if (a.n_group > 1) {
    float* s_val = reinterpret_cast<float*>(s_buf[wid]);
    const int gs = a.E / a.n_group, per = gs / npl;  // lanes per group, where groups are whole lanes
    const bool on_lanes = gs == per * npl && (per & (per - 1)) == 0;
    const bool add = a.group_score == MOE_GROUP_TOP2 && gs > 1;
    float first = -INFINITY, second = -INFINITY;
    const auto value = [&](int j) { return scored ? key_logit(key[j]) : add ? score32(l[j], a.route, st) : l[j]; };
    if (on_lanes) {
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (j < have) top2_add(first, second, value(j));
      for (int o = 1; o < per; o <<= 1) {
        const float f = __shfl_xor_sync(kAll, first, o), s2 = __shfl_xor_sync(kAll, second, o);
        top2_join(first, second, f, s2);
      }
      // lane g takes group g's
      first = __shfl_sync(kAll, first, lane * per & 31);
      second = __shfl_sync(kAll, second, lane * per & 31);
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (j < have) s_val[e0 + j] = value(j);
      __syncwarp();
      // as many lanes per group as there are, a power of two
      int share = 32;
      while (share * a.n_group > 32) share >>= 1;
      if (lane < share * a.n_group) {
        const float* val = s_val + lane / share * gs;
        for (int j = lane & (share - 1); j < gs; j += share) top2_add(first, second, val[j]);
      }
      for (int o = 1; o < share; o <<= 1) {
        const float f = __shfl_xor_sync(kAll, first, o), s2 = __shfl_xor_sync(kAll, second, o);
        top2_join(first, second, f, s2);
      }
      first = __shfl_sync(kAll, first, lane * share & 31);
      second = __shfl_sync(kAll, second, lane * share & 31);
    }
    float score = -INFINITY, err = 0.0f;
    if (lane < a.n_group) {
      score = add ? first + second : first;
      // each key within (bound * p + |key|) ulp, p <= 1; without a bias a single logit is exact, and so is an infinite sum
      if ((scored || add) && fabsf(score) < INFINITY)
        err = kUlp * (fabsf(score) + fabsf(first) + (add ? fabsf(second) : 0.0f) + (add ? 2.0f : 1.0f) * (bound + 1.0f));
    }
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
      const float other = __shfl_sync(kAll, score, g);
      rank += other > score || (other == score && g < lane);
    }
    if (lane >= a.n_group) rank = 64;
    uint32_t kept = __ballot_sync(kAll, rank < a.topk_group);
    // Every kept group against every dropped one: their errors differ with the size of their keys, so it is not enough
    // to look at the two scores next to one another.
    const bool mine_kept = kept >> lane & 1;
    const float low = key_logit(__reduce_min_sync(kAll, order_key(mine_kept ? score - err : INFINITY)));
    const float high =
        key_logit(__reduce_max_sync(kAll, order_key(lane < a.n_group && !mine_kept ? score + err : -INFINITY)));
    const bool clear = above(low, high, 0.0f);
    int g = e0 / gs, left = (g + 1) * gs - e0;  // elements of the lane until the next group
    if ((scored || add) && !clear) {
      // decided by fp64 keys of the elements that may count for a group
      int* list = s_list[wid];
      int n = 0, gg = g, ll = left;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        if (ll == 0) ++gg, ll = gs;
        --ll;
        const float low = __shfl_sync(kAll, add ? second : first, gg & 31);  // lane g holds group g's
        const float v = value(j);
        const bool may = j < have && v >= low - kUlp * (2.0f * bound + 2.0f + fabsf(v) + fabsf(low));
        const uint32_t who = __ballot_sync(kAll, may);
        const int at = n + __popc(who & ((1u << lane) - 1u));
        if (may && at < 32) list[at] = e0 + j;
        n += __popc(who);
      }
      __syncwarp();
      if (n <= 32) kept = groups64(a, row, lane, st.m, n, list);
      else unsure = true;
      __syncwarp();
    }
    if (on_lanes) {
      if (!(kept >> (g & 31) & 1)) {
#pragma unroll
        for (int j = 0; j < NP; ++j) key[j] = 0u;
      }
    } else {
      __syncwarp();  // s_val has been read
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        if (left == 0) ++g, left = gs;
        --left;
        if (!(kept >> (g & 31) & 1)) key[j] = 0u;
      }
    }
  }

  // The k largest, and with a bias the one after them.  Each lane sorts its keys; a round takes the largest head, and
  // the lane that owned it moves its keys up.  Lane r keeps the r-th key and its owner.
  uint32_t* const s_key = reinterpret_cast<uint32_t*>(s_buf[wid]);
#pragma unroll
  for (int j = 0; j < NP; ++j) s_key[j * 32 + lane] = key[j];
  sort_step<NP, 1, 1>(key);
  const int avail = a.n_group > 1 ? a.topk_group * (a.E / a.n_group) : a.E;
  const int rounds = scored && a.k < avail ? a.k + 1 : a.k;
  uint32_t my_key = 0;
  int my_owner = 0;
  const auto pick = [&](int r, uint32_t top) {
    const int owner = __ffs(__ballot_sync(kAll, key[0] == top)) - 1;  // equal keys: the lower lane first
    if (lane == r) my_key = top, my_owner = owner;
    if (lane == owner) {
#pragma unroll
      for (int j = 0; j + 1 < NP; ++j) key[j] = key[j + 1];
      key[NP - 1] = 0u;
    }
  };
  // the element that lane r's choice was: among its owner's equal keys, the one after those of earlier rounds
  const auto element = [&](int n) {
    const uint32_t same = __match_any_sync(kAll, lane < n ? my_key : 0u) & __match_any_sync(kAll, my_owner);
    int skip = __popc(same & ((1u << lane) - 1u)), at = 0;
    bool found = false;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const bool hit = s_key[j * 32 + my_owner] == my_key;
      if (hit && !found && skip-- == 0) at = j, found = true;
    }
    return my_owner * npl + at;
  };
  for (int r = 0; r < rounds; ++r) pick(r, __reduce_max_sync(kAll, key[0]));
  __syncwarp();
  int mine = element(rounds);
  if (lane >= rounds) mine = 0;
  float lg = lane < rounds ? load_logit(a, row + mine) : 0.0f;
  if (scored) {
    const float p = score32(lg, a.route, st);
    const float b = lane < rounds ? __ldg(a.bias + mine) : 0.0f, v = p + b;
    const float err = kUlp * (bound * p + 1.0f + magnitude(v));
    const float v1 = __shfl_down_sync(kAll, v, 1), err1 = __shfl_down_sync(kAll, err, 1);
    const float l1 = __shfl_down_sync(kAll, lg, 1), b1 = __shfl_down_sync(kAll, b, 1);
    const bool same = lg == l1 && b == b1;
    // neighbours of the result, each with its own bound
    bool near = __any_sync(kAll, lane + 1 < a.k && !same && !above(v, v1, err + err1));
    const float vk = __shfl_sync(kAll, v, a.k - 1);
    if (rounds > a.k) {
      // The k-th against all that was not chosen: every one of those lies at or below the next key, but its score, and so
      // its bound, may be anything up to the largest of the row.
      float vn = __shfl_sync(kAll, v, a.k);
      if (__shfl_sync(kAll, (int)same, a.k - 1)) {
        // the next is the k-th's equal in any precision (and of a higher index)
        vn = next_other(a, row, __shfl_sync(kAll, mine, a.k - 1), __shfl_sync(kAll, my_key, a.k - 1), s_key);
      }
      const float most = a.route == MOE_ROUTE_SIGMOID ? 1.0f : st.m == -INFINITY ? 0.0f : fminf(st.inv_sum, 1.0f);
      const float tol = __shfl_sync(kAll, err, a.k - 1) + kUlp * (bound * most + 1.0f + magnitude(vn));
      near |= !above(vk, vn, tol);
    }
    if (near && !unsure) {
      // choices that fp32 cannot order: take more until one is certainly below the k-th, and rank them in fp64
      int n = rounds;
      bool enough = n == avail;
      while (!enough && n < 32) {
        const uint32_t top = __reduce_max_sync(kAll, key[0]);
        if (top == 0) break;
        const float vn = key_logit(top);
        enough = above(vk, vn, kUlp * (2.0f * bound + 2.0f + magnitude(vk) + magnitude(vn)));
        if (!enough) pick(n++, top);
        else break;
      }
      enough |= n < 32;
      if (enough) {
        const int e = element(n);
        mine = rank64(a, row, lane, st.m, n, e, lane < n ? load_logit(a, row + e) : 0.0f);
        if (lane < a.k) lg = load_logit(a, row + mine);
      } else {
        unsure = true;
      }
    }
  }
  if (unsure) {
    mine = select64(a, row, lane, st.m, s_buf[wid]);
    if (lane < a.k) lg = load_logit(a, row + mine);
  }
  const float g = gate(a, lane, lg, st);
  if (lane < a.k) {
    a.ids[(int64_t)t * a.k + lane] = mine;
    a.gates[(int64_t)t * a.k + lane] = g * a.scale;
  }
}

template <int NP>
void launch_np(const RouteArgs& a, unsigned grid, int warps, cudaStream_t s) {
  const int size = a.dtype == MOE_DT_F32 ? 4 : 2;
  const bool vec = a.E == 32 * NP && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
                   (a.T == 1 || a.stride * size % 16 == 0) && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  if constexpr (NP % 8 == 0) {
    if (vec) {
      route_grouped_kernel<NP, true><<<grid, 32 * warps, 0, s>>>(a);
      return;
    }
  }
  route_grouped_kernel<NP, false><<<grid, 32 * warps, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_route_grouped(const RouteArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int npl = (a.E + 31) / 32;
  const int warps = a.T <= 4 * num_sms() ? 1 : 4;  // few tokens: one CTA each
  const unsigned grid = (unsigned)((a.T + warps - 1) / warps);
  note_launch();
  if (npl <= 2) launch_np<2>(a, grid, warps, s);
  else if (npl <= 4) launch_np<4>(a, grid, warps, s);
  else if (npl <= 8) launch_np<8>(a, grid, warps, s);
  else if (npl <= 12) launch_np<12>(a, grid, warps, s);
  else if (npl <= 16) launch_np<16>(a, grid, warps, s);
  else if (npl <= 20) launch_np<20>(a, grid, warps, s);
  else if (npl <= 24) launch_np<24>(a, grid, warps, s);
  else launch_np<32>(a, grid, warps, s);
  return cudaGetLastError();
}

}  // namespace moe
