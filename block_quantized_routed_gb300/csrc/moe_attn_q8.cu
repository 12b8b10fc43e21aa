// Attention of single tokens and verify windows over an 8-bit paged cache.
//
//   a_j = scale * d_j * (q . K_j),   out = sum_j 2^(c a_j) e_j V_j / sum_j 2^(c a_j)
//
// in one pass over the keys with running references (c = log2 e).
//
// What bounds it: memory.  With 8 query heads to a key/value head a key is
// 4 * 8 * D operations for 2 (D + 4) bytes, a sixth of what mma.sync does
// while the bytes arrive, so the products stay on it: its operands are
// registers, and codes become fp16 numbers there (moe_q8.cuh), which tcgen05,
// whose keys and values come from shared memory, would need written back first.
//
// Layout.  Keys are the 16 rows of S^T = K q^T and the 16 terms of out^T = V^T P^T,
// rows of the query (token, head of the key/value head) the 8 columns of a tile,
// NT tiles to an item.  The order of a contraction's terms is free, so a lane
// reads its codes in 16-byte pieces as they lie: it takes 16 consecutive bytes of
// two keys per 64 columns for S, and for the values the same bytes of four
// keys, whose pairs become the halves of an operand register.  Each lane copies
// exactly what it will read itself into a ring of its own (cp.async), so loads
// run several steps ahead without registers or barriers.  P^T is the
// transpose of S^T: one movmatrix per 8 x 8 block.
//
// References.  The weight's factor e_j belongs to the contraction, so it is
// folded into the exponent, P'_j = 2^(c a_j + log2 e_j - m'), with a reference m'
// of its own: fp16 then holds the largest contributions whatever the scales are
// (a first key without values keeps its weight in the sum and takes no range).
// The sum has the reference m.  Both are raised when a score passes them by
// more than 2^8, tested with one vote per 16 keys.
//
// Work split.  Each CTA finds its share of the items' key tiles from cu_q and
// kv_len in a short prologue; an item that is cut leaves partial sums in the
// workspace, and the CTA that arrives last joins them in the order of the keys,
// so results do not depend on timing and no CTA waits for another.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_kv.cuh"
#include "moe_per_device.h"
#include "moe_q8.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxCtas = 320;                     // the workspace holds the partial sums of this many
constexpr size_t kWsHead = 2048;                  // status (16 bytes), a counter per CTA
static_assert(kWsHead >= 16 + 4 * kMaxCtas, "counters");
constexpr int kOver = 2;                          // units of an item besides its key tiles: queries, join of the warps
constexpr int kLeast = 4;                         // units of a CTA at least
constexpr float kLow = -3.0e38f;                  // a reference before any key
constexpr float kGrow = 8.0f;                     // log2 of the growth that raises a reference
constexpr float kLift = 7.0f;                     // log2 of the reference's weight in fp16: at most 2^15 with kGrow
constexpr float kLog2e = 1.44269504088896341f;
constexpr int kPartMax = 4096;                    // elements of an item's accumulator

template <int D_, int NT_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, kRows = 8 * NT;
  static constexpr int W = NT * D <= 256 && D < 256 ? 8 : 4;    // warps
  static constexpr int kTile = 16 * W;                          // keys of a unit
  static constexpr int kStage = 32 * D + 128;                   // 16 keys and values, their scales
  static constexpr int kMisc = kRows * D * 2 + kRows * 16 + W * kRows * 12;
  static constexpr int kStages = std::min(6, (113 * 1024 - 1024 - kMisc) / (W * kStage));  // two CTAs per SM
  static constexpr int kRing = W * kStages * kStage;
  static constexpr int kPitch = D + 4;                          // floats of a row in the join of the warps
  static constexpr int kSmem = kRing + kMisc;
  static constexpr size_t kPartFloats = kPartMax + 3 * 32;      // accumulator; m, m' and sum of each row
  static_assert(kRows * D <= kPartMax && kStages >= 3, "sizes");
  static_assert(W * kRows * kPitch * 4 <= kRing, "the warps' accumulators lie in the ring");
  static_assert((kMaxCtas + 2) * kRows * 4 + 32 * W * 16 <= kRing, "the parts' weights lie in the ring");
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {  // N bytes, zeros if not there
  const int n = there ? N : 0;
  if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // an 8 x 8 block of 16-bit numbers
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// over the 8 lanes that hold the same columns
__device__ __forceinline__ float max_rows(float x) {
  x = fmaxf(x, __shfl_xor_sync(kAll, x, 4));
  x = fmaxf(x, __shfl_xor_sync(kAll, x, 8));
  return fmaxf(x, __shfl_xor_sync(kAll, x, 16));
}
__device__ __forceinline__ float sum_rows(float x) {
  x += __shfl_xor_sync(kAll, x, 4);
  x += __shfl_xor_sync(kAll, x, 8);
  return x + __shfl_xor_sync(kAll, x, 16);
}

// A sequence's items: (key/value head, row tile), each over the key tiles of the whole sequence.
struct Work {
  SeqInfo s;
  int row_tiles, t0, tiles;
  long long units;
};
template <class C>
__device__ __forceinline__ Work work_of(const AttnArgs& a, int G, int b) {
  Work w;
  w.s = seq_info(a.kv, a.cu_q, a.kv_len, a.T, b);
  w.row_tiles = (int)(((long long)w.s.n * G + C::kRows - 1) / C::kRows);
  const int lo = window_lo(w.s.kv - w.s.n + 1, a.window);
  w.t0 = lo / C::kTile;
  w.tiles = max(1, (w.s.kv + C::kTile - 1) / C::kTile - w.t0);
  w.units = (long long)a.kv.Hkv * w.row_tiles * (w.tiles + kOver);
  return w;
}

template <class C>
struct Shared {
  long long scan[C::W], rows[C::W];
  long long total, before;
  int seq, last, over;
};

// writes 4 columns of a row of out
__device__ __forceinline__ void put(const AttnQ8Args& g, int64_t at, float4 v) {
  uint32_t lo, hi;
  if (g.x_dtype == MOE_DT_BF16) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(v.y), "f"(v.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(v.w), "f"(v.z));
  } else {
    lo = half2_of(v.x, v.y);
    hi = half2_of(v.z, v.w);
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.a.out) + at) = make_uint2(lo, hi);
}
__device__ __forceinline__ void fma4(float4& acc, float f, float4 v) {
  acc.x = fmaf(f, v.x, acc.x);
  acc.y = fmaf(f, v.y, acc.y);
  acc.z = fmaf(f, v.z, acc.z);
  acc.w = fmaf(f, v.w, acc.w);
}
// what a row's accumulator is multiplied by, and its lse
template <int FMT>
__device__ __forceinline__ float out_factor(float m, float mv, float sum) {
  return sum == 0.0f ? 0.0f : ex2(mv - m - kLift) / sum * kCodeScale<FMT>;
}
__device__ __forceinline__ float lse_of(float m, float sum) {
  return sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945309f;
}

template <int D, int NT, int FMT>
__global__ void __launch_bounds__(32 * Cfg<D, NT>::W, 2) attn_q8_kernel(const AttnQ8Args ga) {
  using C = Cfg<D, NT>;
  constexpr int W = C::W, kRows = C::kRows, kThreads = 32 * W, kStages = C::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared<C> sh;
  const AttnArgs& a = ga.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int G = a.Hq / a.kv.Hkv;
  uint2* const s_q = reinterpret_cast<uint2*>(smem + C::kRing);                   // [NT][D / 16][lane] operand registers
  float* const s_f = reinterpret_cast<float*>(s_q + kRows * D / 4);               // [row] factor of the scores
  int* const s_lo = reinterpret_cast<int*>(s_f + kRows);                          // [row] keys that it sees
  int* const s_hi = s_lo + kRows;
  float* const s_rf = reinterpret_cast<float*>(s_hi + kRows);                     // [row] factor of its output
  float* const s_m = s_rf + kRows;                                                // [warp][row]
  float* const s_mv = s_m + W * kRows;
  float* const s_l = s_mv + W * kRows;

  // ---- the CTA's share of the units
  {
    const int per = (a.kv.n_seqs + kThreads - 1) / kThreads, b0 = tid * per, b1 = min(a.kv.n_seqs, b0 + per);
    long long mine = 0, rows = 0;
    for (int b = b0; b < b1; ++b) {
      const Work w = work_of<C>(a, G, b);
      if (!w.s.ok) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      mine += w.units;
      rows += w.s.n;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rows += __shfl_xor_sync(kAll, rows, o);
    if (lane == 31) sh.scan[warp] = incl;
    if (lane == 0) sh.rows[warp] = rows;
    __syncthreads();
    long long total = 0, base = 0, all_rows = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) base += sh.scan[w];
      total += sh.scan[w];
      all_rows += sh.rows[w];
    }
    // sequences that share rows (a cu_q out of order): nothing is computed
    if (total == 0 || all_rows > a.T) {
      if (tid == 0 && all_rows > a.T) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      return;
    }
    const long long ctas = min((long long)gridDim.x, max(1ll, total / kLeast));
    if (blockIdx.x >= ctas) return;
    const long long u0 = blockIdx.x * total / ctas;
    long long before = base + incl - mine;
    if (u0 >= before && u0 < before + mine) {
      int b = b0;
      for (;; ++b) {
        const long long u = work_of<C>(a, G, b).units;
        if (u0 < before + u) break;
        before += u;
      }
      sh.seq = b;
      sh.before = before;
      sh.total = total;
    }
    __syncthreads();
  }
  const long long total = sh.total, ctas = min((long long)gridDim.x, max(1ll, total / kLeast));
  const long long u1 = (blockIdx.x + 1) * total / ctas;
  const auto owner = [&](long long u) { return (int)(((u + 1) * ctas - 1) / total); };
  int b = sh.seq;
  long long u = blockIdx.x * total / ctas, base = sh.before;  // the current unit; units before the sequence
  Work w = work_of<C>(a, G, b);
  const uint32_t ring = smem_u32(smem) + warp * (kStages * C::kStage);
  const uint8_t* const ring_p = smem + warp * (kStages * C::kStage);

  while (u < u1) {
    while (u >= base + w.units) {  // the next sequence with tokens
      base += w.units;
      w = work_of<C>(a, G, ++b);
    }
    const int cost = w.tiles + kOver;
    const int item = (int)((u - base) / cost);
    const long long item0 = base + (long long)item * cost, pay0 = item0 + kOver;  // first unit, first key tile
    const int p0 = (int)(max(u, pay0) - pay0), p1 = (int)(min(u1, pay0 + w.tiles) - pay0);
    u = min(u1, item0 + cost);
    if (p0 >= p1) continue;
    const int h = item / w.row_tiles, r0 = (item - h * w.row_tiles) * kRows, nr = min(kRows, w.s.n * G - r0);
    const int off = w.s.kv - w.s.n, tok0 = r0 / G, tok1 = (r0 + nr - 1) / G;
    // keys that some row sees, and those that every row sees (rows behind the last are zeros, and go nowhere)
    const int hi = max(0, off + tok1 + 1), lo = min(hi, window_lo(off + tok0 + 1, a.window));
    const int all_lo = window_lo(off + tok1 + 1, a.window), all_hi = off + tok0 + 1;
    const int from = max(lo, (w.t0 + p0) * C::kTile), to = min(hi, (w.t0 + p1) * C::kTile);
    const int first = from / 16, steps = to > from ? (to + 15) / 16 - first : 0;  // of 16 keys
    const int mine = steps > warp ? (steps - warp + W - 1) / W : 0;               // this warp's: first + warp + W * i

    __syncthreads();  // the last item's join has been read
    // ---- loads of the first steps
    const int32_t* table = a.table + (int64_t)b * a.kv.table_stride;
    const auto page_of = [&](int i) { return i < mine ? __ldg(table + (first + warp + W * i) * 16 / a.kv.page_size) : 0; };
    int next_page = page_of(0);
    const auto issue = [&](int i) {
      if (i < mine) {
        const int key = (first + warp + W * i) * 16, page = next_page;
        const bool there = page >= 0 && page < a.kv.num_pages;
        if (!there && lane == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
        const int slot = key % a.kv.page_size;
        const int64_t pg = there ? page : 0;
        const uint8_t* k = static_cast<const uint8_t*>(a.k_cache) + pg * a.kv.k_page_stride + h * a.kv.k_head_stride +
                           (int64_t)(slot + g) * a.kv.k_row_stride + c * 16;
        const uint32_t dst = ring + (uint32_t)(i % kStages) * C::kStage;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          copy_async<16>(dst + (2 * x) * 512 + lane * 16, k + x * 64, there);
          copy_async<16>(dst + (2 * x + 1) * 512 + lane * 16, k + 8 * a.kv.k_row_stride + x * 64, there);
        }
        constexpr int kV = D == 64 ? 8 : 16;  // bytes of a piece of the values
        const uint8_t* v = static_cast<const uint8_t*>(a.v_cache) + pg * a.kv.v_page_stride + h * a.kv.v_head_stride +
                           (int64_t)(slot + 2 * c) * a.kv.v_row_stride + g * kV;
#pragma unroll
        for (int x = 0; x < (D + 127) / 128; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            copy_async<kV>(dst + 16 * D + ((4 * x + y) * 32 + lane) * kV,
                           v + ((y & 1) + (y >> 1) * 8) * a.kv.v_row_stride + x * 128, there);
        const float* sc = lane < 16 ? ga.sc.k + pg * ga.sc.k_page_stride + h * ga.sc.k_head_stride +
                                          (int64_t)(slot + lane) * ga.sc.k_row_stride
                                    : ga.sc.v + pg * ga.sc.v_page_stride + h * ga.sc.v_head_stride +
                                          (int64_t)(slot + lane - 16) * ga.sc.v_row_stride;
        copy_async<4>(dst + 32 * D + lane * 4, sc, there);
        next_page = page_of(i + 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- queries: fp16 relative to the power of two at the row's largest element, in operand order
    for (int r = warp; r < kRows; r += W) {
      float e[D / 128 > 0 ? D / 128 : 1][4];
      float peak = 0.0f;
      const int R = r0 + r, tok = R / G;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(w.s.q0 + tok) * a.q_stride +
                            (int64_t)(h * G + R - tok * G) * a.q_head_stride;
#pragma unroll
      for (int x = 0; x < (D + 127) / 128; ++x) {
        const int word = x * 32 + lane;
        uint2 v = make_uint2(0, 0);
        if (r < nr && word < D / 4) v = *reinterpret_cast<const uint2*>(src + word * 4);
        if (ga.x_dtype == MOE_DT_BF16) {
          e[x][0] = __uint_as_float(v.x << 16), e[x][1] = __uint_as_float(v.x & 0xffff0000u);
          e[x][2] = __uint_as_float(v.y << 16), e[x][3] = __uint_as_float(v.y & 0xffff0000u);
        } else {
          const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
          const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
          e[x][0] = p.x, e[x][1] = p.y, e[x][2] = q.x, e[x][3] = q.y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) peak = fmaxf(peak, fabsf(e[x][i]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) peak = fmaxf(peak, __shfl_xor_sync(kAll, peak, o));
      int ex = 0;
      if (peak > 0.0f && peak < INFINITY) ex = ilogbf(peak);
      const float up = ldexpf(1.0f, min(14 - ex, 126)), more = ldexpf(1.0f, max(14 - ex - 126, 0));
#pragma unroll
      for (int x = 0; x < (D + 127) / 128; ++x) {
        const int word = x * 32 + lane;
        if (word < D / 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) e[x][i] = e[x][i] * up * more;
          // word: 64 columns, lane's 16, 4 of them
          const int at = ((r >> 3) * (D / 16) + (word >> 4) * 4 + (word & 3)) * 32 + (r & 7) * 4 + (word >> 2 & 3);
          s_q[at] = make_uint2(half2_of(e[x][0], e[x][2]), half2_of(e[x][1], e[x][3]));
        }
      }
      if (lane == 0) {
        s_f[r] = ldexpf(a.scale * kLog2e * kCodeScale<FMT>, ex - 14);
        s_hi[r] = r < nr ? off + tok + 1 : 0;
        s_lo[r] = r < nr ? window_lo(off + tok + 1, a.window) : 0;
      }
    }
    __syncthreads();

    // ---- the warp's steps
    float o[NT][D / 16][4], m[NT][2], mv[NT][2], l[NT][2], f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][t][i] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) m[n][i] = mv[n][i] = kLow, l[n][i] = 0.0f, f[n][i] = s_f[n * 8 + 2 * c + i];
    }
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      issue(i + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const uint8_t* st = ring_p + (i % kStages) * C::kStage;
      const float* sc = reinterpret_cast<const float*>(st + 32 * D);
      const float ks[2] = {sc[g], sc[g + 8]};
      const float lv[2] = {lg2(sc[16 + g]), lg2(sc[24 + g])};
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][x] = 0.0f;
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(st + (2 * x) * 512 + lane * 16);
        const uint4 k1 = *reinterpret_cast<const uint4*>(st + (2 * x + 1) * 512 + lane * 16);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t af[4];
          four_codes<FMT>(w0[y], af[0], af[2]);
          four_codes<FMT>(w1[y], af[1], af[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 q = s_q[(n * (D / 16) + x * 4 + y) * 32 + lane];
            mma(s[n], af, q.x, q.y);
          }
        }
      }
      // scores in powers of two: s of the sum, sv with the value's scale
      float sv[NT][4];
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[n][x] *= f[n][x & 1] * ks[x >> 1];
          sv[n][x] = s[n][x] + lv[x >> 1];
        }
      const int key = (first + warp + W * i) * 16;
      if (key < all_lo || key + 16 > all_hi) {  // some row does not see some key
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = n * 8 + 2 * c + (x & 1), j = key + g + (x >> 1) * 8;
            if (j < s_lo[r] || j >= s_hi[r]) s[n][x] = sv[n][x] = -INFINITY;
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) grow |= s[n][x] > m[n][x & 1] + kGrow || sv[n][x] > mv[n][x & 1] + kGrow;
      if (__any_sync(kAll, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float m1 = fmaxf(m[n][x], max_rows(fmaxf(s[n][x], s[n][x + 2])));
            const float v1 = fmaxf(mv[n][x], max_rows(fmaxf(sv[n][x], sv[n][x + 2])));
            l[n][x] *= ex2(m[n][x] - m1);
            const float fo = ex2(mv[n][x] - v1);
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[n][t][x] *= fo, o[n][t][x + 2] *= fo;
            m[n][x] = m1;
            mv[n][x] = v1;
          }
      }
      uint32_t p[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          l[n][x & 1] += ex2(s[n][x] - m[n][x & 1]);
          sv[n][x] = ex2(sv[n][x] - mv[n][x & 1] + kLift);
        }
        p[n][0] = transposed(half2_of(sv[n][0], sv[n][1]));
        p[n][1] = transposed(half2_of(sv[n][2], sv[n][3]));
      }
      // ---- values: columns 2 u and 2 u + 1 of the lane's bytes are the rows g and g + 8 of an operand
      constexpr int kV = D == 64 ? 8 : 16;
#pragma unroll
      for (int x = 0; x < (D + 127) / 128; ++x) {
        uint32_t v[4][kV / 4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint8_t* src = st + 16 * D + ((4 * x + y) * 32 + lane) * kV;
          if constexpr (kV == 16) {
            const uint4 r = *reinterpret_cast<const uint4*>(src);
            v[y][0] = r.x, v[y][1] = r.y, v[y][2] = r.z, v[y][3] = r.w;
          } else {
            const uint2 r = *reinterpret_cast<const uint2*>(src);
            v[y][0] = r.x, v[y][1] = r.y;
          }
        }
#pragma unroll
        for (int y = 0; y < kV / 4; ++y)
#pragma unroll
          for (int z = 0; z < 2; ++z) {  // bytes 0, 1 and 2, 3 of a word
            constexpr uint32_t kSel[2][2] = {{0x4404, 0x5515}, {0x6626, 0x7737}};
            uint32_t af[4];
            af[0] = upper_codes<FMT>(__byte_perm(v[0][y], v[1][y], kSel[z][0]));
            af[1] = upper_codes<FMT>(__byte_perm(v[0][y], v[1][y], kSel[z][1]));
            af[2] = upper_codes<FMT>(__byte_perm(v[2][y], v[3][y], kSel[z][0]));
            af[3] = upper_codes<FMT>(__byte_perm(v[2][y], v[3][y], kSel[z][1]));
#pragma unroll
            for (int n = 0; n < NT; ++n) mma(o[n][x * 8 + y * 2 + z], af, p[n][0], p[n][1]);
          }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- join of the warps: [warp][row][column] in the ring
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float sum = sum_rows(l[n][x]);
        if (g == 0) {
          const int at = warp * kRows + n * 8 + 2 * c + x;
          s_m[at] = m[n][x], s_mv[at] = mv[n][x], s_l[at] = sum;
        }
      }
    __syncthreads();  // every ring is drained
    float* const acc = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = n * 8 + 2 * c + x;
        if (r < nr) {
          constexpr int kV = D == 64 ? 8 : 16;
          float* dst = acc + (warp * kRows + r) * C::kPitch + g * kV;
#pragma unroll
          for (int t = 0; t < D / 16; t += 2)
            *reinterpret_cast<float4*>(dst + (t / (kV / 2)) * 128 + (t % (kV / 2)) * 2) =
                make_float4(o[n][t][x], o[n][t][x + 2], o[n][t + 1][x], o[n][t + 1][x + 2]);
        }
      }
    const int c0 = owner(pay0), parts = owner(pay0 + w.tiles - 1) - c0 + 1;
    float* const part = reinterpret_cast<float*>(a.ws + kWsHead) +
                        ((size_t)blockIdx.x * 2 + ((int)blockIdx.x == c0 ? 1 : 0)) * C::kPartFloats;
    const auto put_lse = [&](int r, float mm, float sum) {
      if (a.lse) {
        const int R = r0 + r, tok = R / G;
        a.lse[(int64_t)(w.s.q0 + tok) * a.Hq + h * G + R - tok * G] = lse_of(mm, sum);
      }
    };
    const auto row_at = [&](int r) {
      const int R = r0 + r, tok = R / G;
      return (int64_t)(w.s.q0 + tok) * a.o_stride + (int64_t)(h * G + R - tok * G) * a.o_head_stride;
    };
    if (tid < nr) {  // weights of the warps, in place of their references
      float mm = kLow, mmv = kLow, sum = 0.0f;
#pragma unroll
      for (int x = 0; x < W; ++x) mm = fmaxf(mm, s_m[x * kRows + tid]), mmv = fmaxf(mmv, s_mv[x * kRows + tid]);
#pragma unroll
      for (int x = 0; x < W; ++x) {
        sum += s_l[x * kRows + tid] * ex2(s_m[x * kRows + tid] - mm);
        s_mv[x * kRows + tid] = ex2(s_mv[x * kRows + tid] - mmv);
      }
      if (parts == 1) {
        s_rf[tid] = out_factor<FMT>(mm, mmv, sum);
        put_lse(tid, mm, sum);
      } else {
        __stcg(part + kPartMax + tid, mm);
        __stcg(part + kPartMax + 32 + tid, mmv);
        __stcg(part + kPartMax + 64 + tid, sum);
      }
    }
    __syncthreads();
    for (int e = tid; e < nr * (D / 4); e += kThreads) {
      const int r = e / (D / 4), col = e - r * (D / 4);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int x = 0; x < W; ++x)
        fma4(v, s_mv[x * kRows + r], *reinterpret_cast<const float4*>(acc + (x * kRows + r) * C::kPitch + col * 4));
      if (parts == 1) {
        const float rf = s_rf[r];
        put(ga, row_at(r) + col * 4, make_float4(v.x * rf, v.y * rf, v.z * rf, v.w * rf));
      } else {
        __stcg(reinterpret_cast<float4*>(part) + e, v);
      }
    }
    if (parts == 1) continue;

    // ---- an item of several CTAs: the last to arrive joins its parts
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      unsigned* counter = reinterpret_cast<unsigned*>(a.ws + 16) + c0;
      sh.last = atomicInc(counter, (unsigned)parts - 1) == (unsigned)parts - 1;  // wraps to 0 behind the last
      __threadfence();
    }
    __syncthreads();
    if (!sh.last) continue;
    const float* const part0 = reinterpret_cast<const float*>(a.ws + kWsHead);
    const auto part_of = [&](int p) { return part0 + ((size_t)(c0 + p) * 2 + (p == 0 ? 1 : 0)) * C::kPartFloats; };
    float* const wgt = reinterpret_cast<float*>(smem);  // [part][nr]
    for (int r = warp; r < nr; r += W) {                // a warp per row, a lane per part
      float mm = kLow, mmv = kLow, sum = 0.0f;
      for (int p = lane; p < parts; p += 32) {
        mm = fmaxf(mm, __ldcg(part_of(p) + kPartMax + r));
        mmv = fmaxf(mmv, __ldcg(part_of(p) + kPartMax + 32 + r));
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) {
        mm = fmaxf(mm, __shfl_xor_sync(kAll, mm, x));
        mmv = fmaxf(mmv, __shfl_xor_sync(kAll, mmv, x));
      }
      for (int p = lane; p < parts; p += 32) {
        sum += __ldcg(part_of(p) + kPartMax + 64 + r) * ex2(__ldcg(part_of(p) + kPartMax + r) - mm);
        wgt[p * nr + r] = ex2(__ldcg(part_of(p) + kPartMax + 32 + r) - mmv);
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(kAll, sum, x);
      if (lane == 0) {
        s_rf[r] = out_factor<FMT>(mm, mmv, sum);
        put_lse(r, mm, sum);
      }
    }
    __syncthreads();
    const int n = nr * (D / 4);
    int teams = 1;  // teams of threads share the parts where there are few vectors
    while (teams * 2 * n <= kThreads && teams * 2 <= parts) teams *= 2;
    const int width = kThreads / teams, team = tid / width;
    float4* const red = reinterpret_cast<float4*>(smem + C::kRing - kThreads * 16);
    for (int e0 = 0; e0 < n; e0 += width) {  // (once where there are teams)
      const int e = e0 + tid - team * width;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (e < n) {
        const int r = e / (D / 4);
#pragma unroll 8
        for (int p = team; p < parts; p += teams) fma4(v, wgt[p * nr + r], __ldcg(reinterpret_cast<const float4*>(part_of(p)) + e));
      }
      if (teams > 1) {
        red[tid] = v;
        __syncthreads();
        if (team == 0)
          for (int x = 1; x < teams; ++x) fma4(v, 1.0f, red[tid + x * width]);
      }
      if (team == 0 && e < n) {
        const int r = e / (D / 4), col = e - r * (D / 4);
        const float rf = s_rf[r];
        put(ga, row_at(r) + col * 4, make_float4(v.x * rf, v.y * rf, v.z * rf, v.w * rf));
      }
    }
  }
}

template <int D, int NT, int FMT>
cudaError_t launch_t(const AttnQ8Args& a, cudaStream_t s) {
  using C = Cfg<D, NT>;
  auto kern = attn_q8_kernel<D, NT, FMT>;
  static PerDevice opted;
  cudaError_t err = cudaSuccess;
  opted([&](int) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    return err == cudaSuccess ? 1 : 0;
  });
  if (err != cudaSuccess) return err;
  note_launch();
  kern<<<std::min(2 * num_sms(), kMaxCtas), 32 * C::W, C::kSmem, s>>>(a);
  return cudaGetLastError();
}
template <int D, int FMT>
cudaError_t launch_rows(const AttnQ8Args& g, cudaStream_t s) {
  // Rows of an item: those of a sequence of the mean number of new tokens, and a third more, since the lengths of
  // verify windows differ and a window that does not fit reads its keys twice.
  const int64_t mean = (g.a.T + (int64_t)g.a.kv.n_seqs - 1) / g.a.kv.n_seqs, rows = g.a.Hq / g.a.kv.Hkv * mean;
  const int64_t want = mean > 1 ? rows + rows / 3 : rows;
  if (want <= 8) return launch_t<D, 1, FMT>(g, s);
  if (D == 256 || want <= 16) return launch_t<D, 2, FMT>(g, s);
  return launch_t<D, D == 256 ? 2 : 4, FMT>(g, s);
}
template <int D>
cudaError_t launch_fmt(const AttnQ8Args& g, cudaStream_t s) {
  return g.a.kv.dtype == MOE_DT_E4M3 ? launch_rows<D, MOE_DT_E4M3>(g, s) : launch_rows<D, MOE_DT_INT8>(g, s);
}

}  // namespace

bool attn_q8_tensor_core(const AttnQ8Args& g) {
  const moe_kv_desc& kv = g.a.kv;
  const int64_t strides[] = {kv.k_page_stride, kv.k_row_stride, kv.k_head_stride,
                             kv.v_page_stride, kv.v_row_stride, kv.v_head_stride};
  for (int64_t v : strides)
    if (v % 16) return false;
  return (kv.D == 64 || kv.D == 128 || kv.D == 256) && kv.page_size % 16 == 0 &&
         reinterpret_cast<uintptr_t>(g.a.k_cache) % 16 == 0 && reinterpret_cast<uintptr_t>(g.a.v_cache) % 16 == 0;
}

size_t attn_q8_workspace(int, int, int D) {
  if (D != 64 && D != 128 && D != 256) return 256;
  return kWsHead + (size_t)kMaxCtas * 2 * Cfg<64, 1>::kPartFloats * 4;
}

cudaError_t launch_attn_q8(const AttnQ8Args& g, cudaStream_t s) {
  if (g.a.T == 0) return cudaSuccess;
  if (g.a.kv.D == 64) return launch_fmt<64>(g, s);
  return g.a.kv.D == 128 ? launch_fmt<128>(g, s) : launch_fmt<256>(g, s);
}

}  // namespace moe
