// Attention of single tokens and verify windows over an 8-bit paged cache.
//
//   a_j = scale * d_j * (q . K_j),   out = sum_j 2^(c a_j) e_j V_j / sum_j 2^(c a_j)
//
// in one pass over the keys with running references (c = log2 e).
//
// What bounds it: for single tokens memory.  With 8 query heads to a key/value
// head a key is 4 * 8 * D operations for 2 (D + 4) bytes, a sixth of what mma.sync
// does while the bytes arrive, so the products stay on it: its operands are
// registers, and codes become fp16 numbers there (moe_q8.cuh), which tcgen05,
// whose keys and values come from shared memory, would need written back first.
// That reason ends with 8 rows: at 32, four tokens of such heads, a key costs two
// thirds of mma.sync's rate and four times the exponentials, and more rows read
// their keys again.  16 sequences of 4096 keys (32 heads over 4 of 128): 1, 4, 8
// and 16 new tokens each 21, 43, 66 and 115 us.
//
// Layout.  Keys are the 16 rows of S^T = K q^T and the 16 terms of out^T = V^T P^T,
// rows of the query (token, head of the key/value head) the 8 columns of a tile,
// NT tiles to an item.  A CTA takes a tile of keys at a time, 16 to each warp: TMA
// boxes of their codes, found through the page table, land in a ring of tiles,
// and the warp that is the last to finish a tile asks for the one that takes its
// place, so nobody waits but for data.  The order of a contraction's terms is
// free, so a lane reads codes in 16-byte pieces as they lie: pieces of two keys
// for S, and for the values the same piece of four keys, whose pairs become the
// halves of an operand register; the boxes' swizzle keeps both reads free of bank
// conflicts.  P^T is the transpose of S^T: one movmatrix per 8 x 8 block.
//
// References.  The weight's factor e_j belongs to the contraction, so it is
// folded into the exponent, P'_j = 2^(c a_j + log2 e_j - m'), with a reference m'
// of its own: fp16 then holds the largest contributions whatever the scales are
// (a first key without values keeps its weight in the sum and takes no range).
// The sum has the reference m.  Both are raised when a score passes them by
// more than 2^8, tested with one vote per 16 keys.
//
// Work split.  Each CTA finds its share of the items' key tiles from cu_q and
// kv_len in a short prologue: items in equal parts, a part to a CTA, or, where
// that leaves the CTAs uneven or items are many, even shares of all tiles laid
// end to end.  An item of several CTAs leaves partial sums in the workspace, and
// the CTA that arrives last joins them in the order of the keys, so results do
// not depend on timing and no CTA waits for another.
//
// What it measured (e4m3): four tokens over up to 131072 keys each (64 heads over
// 8 of 128) 103 to 113 us, 5.1 to 5.6 TB/s; 48 over up to 8192 keys (32 over 4 of
// 128) 48 us, 4.7 TB/s: tile by tile about 7, besides 5 us to the first and 4 from
// the last; one over 777 keys 11.5 us, latency: of a CTA's clocks a third go by
// until its first boxes are asked for, through cu_q, the page table and
// instructions that are fetched for the first time, and half in the joins of its
// warps and of the parts, through global memory.
#include <algorithm>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_kv.cuh"
#include "moe_overlap.cuh"
#include "moe_per_device.h"
#include "moe_q8.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxCtas = 320;                     // the workspace holds the partial sums of this many
constexpr size_t kWsHead = 2048;                  // status (16 bytes), a counter per CTA
static_assert(kWsHead >= 16 + 4 * kMaxCtas, "counters");
constexpr int kOver = 4;                          // units of an item besides its key tiles: queries, join of the warps
constexpr int kLeast = 2;                         // key tiles of a CTA at least
constexpr int kCut = 4;                           // what even shares cost besides: two cut items a CTA
constexpr float kLow = -3.0e38f;                  // a reference before any key
constexpr float kGrow = 8.0f;                     // log2 of the growth that raises a reference
constexpr float kLift = 7.0f;                     // log2 of the reference's weight in fp16: at most 2^15 with kGrow
constexpr long long kWaitCycles = 2000000000ll;  // ~1 s at 2 GHz
constexpr float kLog2e = 1.44269504088896341f;
constexpr int kPartMax = 4096;                    // elements of an item's accumulator

template <int D_, int NT_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, kRows = 8 * NT;
  static constexpr int W = NT * D <= 128 ? 8 : 4;               // warps: 128 or 256 registers a thread, two CTAs per SM
  static constexpr int kTile = 16 * W;                          // keys of a unit
  static constexpr int kLine = D < 128 ? D : 128, kHalves = D / kLine;  // copied boxes have lines of up to 128 bytes
  static constexpr int kPlane = kTile * kLine;                  // a tile's lines of one half of the keys or values
  static constexpr int kStage = 2 * kHalves * kPlane;           // keys, then values
  static constexpr int kScales = 128;                           // of a warp and stage: scales of 16 keys, then of their values
  static constexpr int kMisc = kRows * D * 2 + kRows * 16 + W * kRows * 12;
  static constexpr int kStages = std::min(6, (113 * 1024 - 2048 - kMisc) / (kStage + W * kScales + 16));  // two CTAs per SM
  static constexpr int kRing = kStages * kStage;
  static constexpr int kSmemScales = kRing, kSmemBars = kSmemScales + W * kStages * kScales;
  static constexpr int kSmemMisc = kSmemBars + kStages * 16;    // a barrier and a count of warps per stage
  static constexpr int kSmem = kSmemMisc + kMisc + 1024;        // (the ring starts on a 1024-byte boundary)
  static constexpr int kPitch = D + 4;                          // floats of a row in the join of the warps
  static constexpr size_t kPartFloats = kPartMax + 3 * 32;      // accumulator; m, m' and sum of each row
  static_assert(kRows * D <= kPartMax && kStages >= 3, "sizes");
  static_assert(W * kRows * kPitch * 4 <= kRing, "the warps' accumulators lie in the ring");
  static_assert((kMaxCtas + 2) * kRows * 4 + 32 * W * 16 <= kRing, "the parts' weights lie in the ring");
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int row, int head, int page,
                                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src, bool there) {  // zeros if not there
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
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
  int row_tiles, items, t0, tiles;
  __device__ __forceinline__ int units() const { return items * (tiles + kOver); }  // of a call fewer than 2^31: attn_q8_fits
};
template <class C>
__device__ __forceinline__ Work work_of(const AttnArgs& a, int G, int b) {
  Work w;
  w.s = seq_info(a.kv, a.cu_q, a.kv_len, a.T, b);
  w.row_tiles = (w.s.n * G + C::kRows - 1) / C::kRows;
  w.items = a.kv.Hkv * w.row_tiles;
  const int lo = window_lo(w.s.kv - w.s.n + 1, a.window);
  w.t0 = lo / C::kTile;
  w.tiles = max(1, (w.s.kv + C::kTile - 1) / C::kTile - w.t0);
  return w;
}

constexpr int kTries = 4;  // sizes of a part that are tried, in steps of an eighth
template <class C>
struct Shared {
  int scan[C::W], items[C::W], ctas[C::W][kTries];
  long long rows[C::W];
  int seq, before, last;
  Work work;
  volatile int abort;
};

// a / b of numbers that are not negative, quick where a < 2^20: the quotient of a + 1/2 lies at least 1 / (2 b) from a
// whole number, more than its error.
__device__ __forceinline__ int quotient(int a, int b) { return a < 1 << 20 ? (int)__fdividef((float)a + 0.5f, (float)b) : a / b; }
__device__ __forceinline__ int quotient(long long a, int b) {
  return a < 1 << 20 ? quotient((int)a, b) : (int)(a / b);
}

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
// What a row's accumulator is multiplied by, one after the other: 2^(mv - m - kLift) / sum in two halves, because the
// power alone is no fp32 number where all scales are small (2^-126 is the least) though the product is one.
__device__ __forceinline__ void out_factors(float m, float mv, float sum, float& first, float& second) {
  first = ex2((mv - m - kLift) * 0.5f);
  second = sum == 0.0f ? 0.0f : first / sum;
}
__device__ __forceinline__ float4 times(float4 v, float first, float second) {
  return make_float4(v.x * first * second, v.y * first * second, v.z * first * second, v.w * first * second);
}
// a row's lse
__device__ __forceinline__ float lse_of(float m, float sum) {
  return sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945309f;
}

template <int D, int NT, int FMT>
__global__ void __launch_bounds__(32 * Cfg<D, NT>::W, 2) attn_q8_kernel(const AttnQ8Args ga, const __grid_constant__ CUtensorMap km,
                                                                        const __grid_constant__ CUtensorMap vm) {
  using C = Cfg<D, NT>;
  constexpr int W = C::W, kRows = C::kRows, kThreads = 32 * W, kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023);  // the swizzled boxes start on 1024-byte boundaries
  __shared__ Shared<C> sh;
  const AttnArgs& a = ga.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int G = ga.G;
  uint2* const s_q = reinterpret_cast<uint2*>(smem + C::kSmemMisc);               // [NT][D / 16][lane] operand registers
  float* const s_f = reinterpret_cast<float*>(s_q + kRows * D / 4);               // [row] factor of the scores; in a join, s_rf's second
  int* const s_lo = reinterpret_cast<int*>(s_f + kRows);                          // [row] keys that it sees
  int* const s_hi = s_lo + kRows;
  float* const s_rf = reinterpret_cast<float*>(s_hi + kRows);                     // [row] factor of its output
  float* const s_m = s_rf + kRows;                                                // [warp][row]
  float* const s_mv = s_m + W * kRows;
  float* const s_l = s_mv + W * kRows;

  const uint32_t ring = smem_u32(smem), bars = ring + C::kSmemBars;
  int* const s_done = reinterpret_cast<int*>(smem + C::kSmemBars + kStages * 8);  // [stage] warps that have finished with it
  if (tid < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tid ? &vm : &km)) : "memory");
  if (tid < kStages) {
    bar_init(bars + tid * 8);
    s_done[tid] = 0;
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (tid == 0) sh.abort = 0;
  let_next_start();
  wait_for_previous();

  // ---- the CTA's share of the work: parts of `size` key tiles, or (size 0) the units from u to u1 of `total` on `ctas` CTAs
  int size = 0, total = 0, ctas = gridDim.x, u = 0, u1 = 1;
  {
    const int per = (a.kv.n_seqs + kThreads - 1) / kThreads, b0 = tid * per, b1 = min(a.kv.n_seqs, b0 + per);
    Work mine{};  // of the thread's (last) sequence
    long long rows = 0;
    int items = 0, units = 0;
    for (int b = b0; b < b1; ++b) {
      mine = work_of<C>(a, G, b);
      if (!mine.s.ok) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      rows += mine.s.n;
      items += mine.items;
      units += mine.units();
    }
    // sums over the threads before, in the order of the sequences, and over all
    const auto scan = [&](int x, int& all) {
      int incl = x;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      const int y = lane < W ? sh.scan[lane] : 0;
      all = __reduce_add_sync(kAll, y);
      const int before = incl - x + __reduce_add_sync(kAll, lane < warp ? y : 0);
      return before;
    };
    rows = min(rows, (long long)a.T + 1);
    rows = ((long long)__reduce_add_sync(kAll, (unsigned)(rows >> 16)) << 16) + __reduce_add_sync(kAll, (unsigned)(rows & 0xffff));
    const int warp_items = __reduce_add_sync(kAll, items);
    if (lane == 0) {
      sh.items[warp] = warp_items;
      sh.rows[warp] = rows;
    }
    int before = scan(units, total);
    const int all_items = __reduce_add_sync(kAll, lane < W ? sh.items[lane] : 0);
    long long all_rows = 0;
#pragma unroll 1
    for (int x = 0; x < W; ++x) all_rows += sh.rows[x];
    // sequences that share rows (a cu_q out of order): nothing is computed
    if (total == 0 || all_rows > a.T) {
      if (tid == 0 && all_rows > a.T) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      return;
    }
    // Equal parts: the smallest of a few sizes for which there are CTAs enough, if it is not much larger than an even share.
    if (all_items <= ctas && per == 1) {
      const int shared = min(ctas, max(1, total / (kLeast + kOver)));  // CTAs of even shares
      const int least = max(kLeast, (total - kOver * all_items + ctas - 1) / ctas);
      const auto tried = [&](int k) { return least + (least * k + 7) / 8; };
#pragma unroll
      for (int k = 0; k < kTries; ++k) {
        const int sum = __reduce_add_sync(kAll, items * quotient(mine.tiles + tried(k) - 1, tried(k)));
        if (lane == 0) sh.ctas[warp][k] = sum;
      }
      __syncthreads();
      const int even = quotient(total, shared) + kCut - kOver;
#pragma unroll
      for (int k = kTries - 1; k >= 0; --k) {
        const int sum = __reduce_add_sync(kAll, lane < W ? sh.ctas[lane][k] : 0);
        if (sum <= ctas && tried(k) <= even) size = tried(k);
      }
    }
    if (size) {
      units = items * quotient(mine.tiles + size - 1, size);
      before = scan(units, total);
      u = blockIdx.x;
      if (u >= total) return;
    } else {
      ctas = min(ctas, max(1, total / (kLeast + kOver)));
      if ((int)blockIdx.x >= ctas) return;
      u = quotient((long long)blockIdx.x * total, ctas);
      u1 = quotient((long long)(blockIdx.x + 1) * total, ctas);
    }
    if (u >= before && u < before + units) {  // this thread has the sequence of the CTA's first unit (of its part)
      int b = b0;
      if (per > 1) {
        for (;; ++b) {
          mine = work_of<C>(a, G, b);
          if (u < before + mine.units()) break;
          before += mine.units();
        }
      }
      sh.seq = b;
      sh.before = before;
      sh.work = mine;
    }
    __syncthreads();
  }
  const auto owner = [&](int x) { return quotient(((long long)x + 1) * ctas - 1, total); };
  int b = sh.seq, base = sh.before;  // units before the sequence
  Work w = sh.work;
  const float* const scales_p = reinterpret_cast<const float*>(smem + C::kSmemScales + warp * (kStages * C::kScales));
  const uint32_t scales = smem_u32(scales_p);
  // keys of a box: a power of two that divides a page and a tile
  const int box = min(C::kTile, a.kv.page_size & -a.kv.page_size), boxes = C::kTile / box, batch = 32 / boxes;
  int got = 0;              // the stage that is read next
  uint32_t parity = 0;      // of its barrier

  for (bool more = true; more;) {
    int item, p0, p1, c0, parts;  // the item and its tiles of this CTA; the first of its CTAs, and how many
    if (size) {
      parts = quotient(w.tiles + size - 1, size);
      item = quotient(u - base, parts);
      c0 = base + item * parts;
      const int each = quotient(w.tiles + parts - 1, parts);
      p0 = (u - c0) * each;
      p1 = min(w.tiles, p0 + each);
      more = false;
    } else {
      while (u - base >= w.units()) {  // the next sequence with tokens
        base += w.units();
        w = work_of<C>(a, G, ++b);
      }
      const int cost = w.tiles + kOver;
      item = quotient(u - base, cost);
      const int pay0 = base + item * cost + kOver;  // the unit of the first key tile
      p0 = max(u, pay0) - pay0;
      p1 = min(u1, pay0 + w.tiles) - pay0;
      u = min(u1, pay0 + w.tiles);
      more = u < u1;
      if (p0 >= p1) continue;
      c0 = owner(pay0);
      parts = owner(pay0 + w.tiles - 1) - c0 + 1;
    }
    const int h = w.row_tiles == 1 ? item : quotient(item, w.row_tiles), r0 = (item - h * w.row_tiles) * kRows;
    const int nr = min(kRows, w.s.n * G - r0);
    const int off = w.s.kv - w.s.n, tok0 = quotient(r0, G), tok1 = quotient(r0 + nr - 1, G);
    // keys that some row sees, and those that every row sees (rows behind the last are zeros, and go nowhere)
    const int hi = max(0, off + tok1 + 1), lo = min(hi, window_lo(off + tok0 + 1, a.window));
    const int all_lo = window_lo(off + tok1 + 1, a.window), all_hi = off + tok0 + 1;
    const int from = max(lo, (w.t0 + p0) * C::kTile), to = min(hi, (w.t0 + p1) * C::kTile);
    const int first = from / C::kTile;                                                   // key tile
    const int tiles = to > from && !sh.abort ? (to + C::kTile - 1) / C::kTile - first : 0;

    // ---- pages of the first tiles, a box to a lane, and the query rows: all asked for at once
    const int32_t* const table = a.table + (int64_t)b * a.kv.table_stride;
    int page, slot;  // of box `lane` of the current batch of tiles; page -1: reads as zeros
    const auto look_up = [&](int i) {
      const int tile = i + lane / boxes;
      const uint32_t key = (uint32_t)(first + tile) * C::kTile + (lane % boxes) * box, entry = key / (uint32_t)a.kv.page_size;
      slot = (int)(key - entry * a.kv.page_size);
      page = -1;
      if (tile < tiles && key < (uint32_t)to && key + box > (uint32_t)from) {  // (some of its keys are seen)
        page = __ldg(table + entry);
        if (page < 0 || page >= a.kv.num_pages) {
          if (warp == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
          page = -1;
        }
      }
    };
    look_up(0);
    // lane r: where row r of the queries lies; a pass of a warp takes one row, two where a row is half a warp's words
    constexpr int kWide = D == 64 ? 16 : 32, kRowsOfPass = 32 / kWide, kWords = (D + 127) / 128;
    constexpr int kPasses = kRows / (W * kRowsOfPass) > 0 ? kRows / (W * kRowsOfPass) : 1;
    const int my_tok = quotient(r0 + min(lane, nr - 1), G);
    const int64_t my_row = (int64_t)(w.s.q0 + my_tok) * a.q_stride +
                           (int64_t)(h * G + r0 + min(lane, nr - 1) - my_tok * G) * a.q_head_stride;
    const auto row_of = [&](int y) { return (y * W + warp) * kRowsOfPass + lane / kWide; };
    uint2 qw[kPasses][kWords];
#pragma unroll
    for (int y = 0; y < kPasses; ++y) {
      const int r = row_of(y);
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + __shfl_sync(kAll, my_row, r);
#pragma unroll
      for (int x = 0; x < kWords; ++x) {
        qw[y][x] = make_uint2(0, 0);
        if (r < nr) qw[y][x] = *reinterpret_cast<const uint2*>(src + (x * 32 + lane % kWide) * 4);
      }
    }
    fence_proxy();
    __syncthreads();  // the last item's join has been read
    // ---- loads of the first tiles
    const bool of_keys = lane < 16;
    const float* const sc0 = of_keys ? ga.sc.k + h * ga.sc.k_head_stride : ga.sc.v + h * ga.sc.v_head_stride;
    const int64_t sc_page = of_keys ? ga.sc.k_page_stride : ga.sc.v_page_stride;
    const int64_t sc_row = of_keys ? ga.sc.k_row_stride : ga.sc.v_row_stride;
    const int my_box = warp * 16 / box, my_line = warp * 16 % box + (lane & 15);
    // the warp's scales of tile i into stage st
    const auto ask_scales = [&](int i, int st) {
      const int from_lane = i % batch * boxes + my_box;
      const int pg = __shfl_sync(kAll, page, from_lane), at = __shfl_sync(kAll, slot, from_lane) + my_line;
      copy_async4(scales + st * C::kScales + lane * 4, sc0 + max(pg, 0) * sc_page + at * sc_row, pg >= 0);
    };
    // the codes of tile i into stage st: a box to a lane
    const auto ask_codes = [&](int i, int st) {
      const int which = lane % boxes, plane = lane / boxes;
      const int from_lane = i % batch * boxes + which;
      const int pg = __shfl_sync(kAll, page, from_lane), at = __shfl_sync(kAll, slot, from_lane);
      const uint32_t bar = bars + st * 8;
      if (lane == 0) bar_expect(bar, C::kStage);
      __syncwarp();
      if (plane < 2 * C::kHalves) {
        const bool values = plane >= C::kHalves;
        tma_4d(ring + st * C::kStage + plane * C::kPlane + which * box * C::kLine, values ? &vm : &km,
               (values ? plane - C::kHalves : plane) * 128, at, h, pg >= 0 ? pg : a.kv.num_pages, bar);
      }
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) {
      if (i < tiles) {
        const int st = got + i < kStages ? got + i : got + i - kStages;
        if (i && i % batch == 0) look_up(i);
        if (warp == i % W) ask_codes(i, st);
        ask_scales(i, st);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }

    // ---- queries: fp16 relative to the power of two at the row's largest element, in operand order
    float e[kPasses][kWords][4], peak[kPasses];
#pragma unroll
    for (int y = 0; y < kPasses; ++y) {
      peak[y] = 0.0f;
#pragma unroll
      for (int x = 0; x < kWords; ++x) {
        const uint2 v = qw[y][x];
        if (ga.x_dtype == MOE_DT_BF16) {
          e[y][x][0] = __uint_as_float(v.x << 16), e[y][x][1] = __uint_as_float(v.x & 0xffff0000u);
          e[y][x][2] = __uint_as_float(v.y << 16), e[y][x][3] = __uint_as_float(v.y & 0xffff0000u);
        } else {
          const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
          const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
          e[y][x][0] = p.x, e[y][x][1] = p.y, e[y][x][2] = q.x, e[y][x][3] = q.y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) peak[y] = fmaxf(peak[y], fabsf(e[y][x][i]));
      }
    }
#pragma unroll
    for (int o = kWide / 2; o > 0; o >>= 1)
#pragma unroll
      for (int y = 0; y < kPasses; ++y) peak[y] = fmaxf(peak[y], __shfl_xor_sync(kAll, peak[y], o));
#pragma unroll
    for (int y = 0; y < kPasses; ++y) {
      const int r = row_of(y);
      if (r >= kRows) break;  // (more warps than rows)
      // its exponent, where 2^-126 times it is a number; the largest element becomes 2^14 .. 2^15
      const uint32_t ex = min(max(__float_as_uint(peak[y]) >> 23, 15u), 254u);
      const float up = __uint_as_float((268 - ex) << 23);
#pragma unroll
      for (int x = 0; x < kWords; ++x) {
        const int word = x * 32 + lane % kWide;
        float* v = e[y][x];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= up;
        // a line's pieces of 16 columns go to the lanes c in order (two each, where a line has 8), 4 columns at a time
        const int piece = word >> 2 & (C::kLine / 16 - 1), of = D == 64 ? piece : piece >> 1;
        const int step = (D == 64 ? 0 : (word >> 5) * 8 + (piece & 1) * 4) + (word & 3);
        s_q[((r >> 3) * (D / 16) + step) * 32 + (r & 7) * 4 + of] =
            FMT == MOE_DT_E4M3 ? make_uint2(half2_of(v[0], v[1]), half2_of(v[2], v[3]))
                               : make_uint2(half2_of(v[0], v[2]), half2_of(v[1], v[3]));
      }
      if (lane % kWide == 0) s_f[r] = a.scale * kLog2e * __uint_as_float((ex - 14) << 23);
    }
    if (warp == W - 1 && lane < kRows) {
      s_hi[lane] = lane < nr ? off + my_tok + 1 : 0;
      s_lo[lane] = lane < nr ? window_lo(off + my_tok + 1, a.window) : 0;
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
    for (int i = 0; i < tiles; ++i) {
      const int st_no = got;
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      if (!bar_try(bars + got * 8, parity)) {
        const long long t0 = clock64();
        while (!sh.abort && !bar_try(bars + got * 8, parity))
          if (clock64() - t0 > kWaitCycles) {
            sh.abort = 1;
            set_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
          }
      }
      __syncwarp();  // the scales that other lanes asked for are there too (a vote orders no memory)
      if (__any_sync(kAll, sh.abort)) break;  // given up: what this call computes is void
      if (++got == kStages) got = 0, parity ^= 1;
      const int key = (first + i) * C::kTile + warp * 16;
      if (key < to && key + 16 > from) {
        const uint8_t* const st = smem + st_no * C::kStage + warp * 16 * C::kLine;
        const float* const sc = scales_p + st_no * (C::kScales / 4);
        const float ks[2] = {sc[g], sc[g + 8]};
        const float lv[2] = {lg2(sc[16 + g]), lg2(sc[24 + g])};
        constexpr int kChains = NT == 1 ? 2 : 1;  // sums that do not wait for one another
        float s[NT][4], s2[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s2[x] = 0.0f;
#pragma unroll
          for (int n = 0; n < NT; ++n) s[n][x] = 0.0f;
        }
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          // lines g and g + 8, the same place in both: the swizzle repeats after 8 lines
          const uint8_t* src = st + (x >> 1) * C::kPlane + g * C::kLine +
                               ((D == 64 ? c ^ (g >> 1 & 3) : (2 * c + (x & 1)) ^ g) << 4);
          const uint4 k0 = *reinterpret_cast<const uint4*>(src);
          const uint4 k1 = *reinterpret_cast<const uint4*>(src + 8 * C::kLine);
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t af[4];
            four_codes<FMT>(w0[y], af[0], af[2]);
            four_codes<FMT>(w1[y], af[1], af[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint2 q = s_q[(n * (D / 16) + x * 4 + y) * 32 + lane];
              mma(kChains == 2 && (y & 1) ? s2 : s[n], af, q.x, q.y);
            }
          }
        }
        if constexpr (kChains == 2) {
#pragma unroll
          for (int x = 0; x < 4; ++x) s[0][x] += s2[x];
        }
        // a lane's piece of the values of its four keys
        constexpr int kV = D == 64 ? 8 : 16;
        uint32_t v[C::kHalves][4][kV / 4];
#pragma unroll
        for (int x = 0; x < C::kHalves; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int line = 2 * c + (y & 1);  // and its swizzle; line + 8 has the same
            const uint8_t* src = st + (C::kHalves + x) * C::kPlane + (line + (y >> 1) * 8) * C::kLine;
            if constexpr (kV == 16) {
              const uint4 r = *reinterpret_cast<const uint4*>(src + ((g ^ line) << 4));
              v[x][y][0] = r.x, v[x][y][1] = r.y, v[x][y][2] = r.z, v[x][y][3] = r.w;
            } else {
              const uint2 r = *reinterpret_cast<const uint2*>(src + (((g >> 1) ^ (line >> 1)) << 4) + (g & 1) * 8);
              v[x][y][0] = r.x, v[x][y][1] = r.y;
            }
          }
        // scores in powers of two: s of the sum, sv with the value's scale
        float sv[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            s[n][x] *= f[n][x & 1] * ks[x >> 1];
            sv[n][x] = s[n][x] + lv[x >> 1];
          }
        const bool partly = key < all_lo || key + 16 > all_hi;  // some row does not see some key
        if (partly) {
          uint32_t nan_keys = 0;  // of the 16: a value's code is e4m3's NaN, which only the rows that see it may meet
          if constexpr (FMT == MOE_DT_E4M3) {
#pragma unroll
            for (int x = 0; x < C::kHalves; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int z = 0; z < kV / 4; ++z)
                  if (__vcmpeq4(v[x][y][z] & 0x7f7f7f7fu, 0x7f7f7f7fu)) nan_keys |= 1u << (2 * c + (y & 1) + (y >> 1) * 8);
            nan_keys = __reduce_or_sync(kAll, nan_keys);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int r = n * 8 + 2 * c + (x & 1), j = key + g + (x >> 1) * 8;
              if (j < s_lo[r] || j >= s_hi[r]) s[n][x] = sv[n][x] = -INFINITY;
              else if (nan_keys >> (j - key) & 1) sv[n][x] = NAN;
            }
        }
        bool grow = false;
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
        // columns 2 z and 2 z + 1 of the lane's piece are the rows g and g + 8 of an operand
        const auto values = [&](auto finite) {
#pragma unroll
          for (int x = 0; x < C::kHalves; ++x)
#pragma unroll
            for (int y = 0; y < kV / 4; ++y) {
              uint32_t af[2][4];
              if constexpr (decltype(finite)::value) {
                two_keys_finite<FMT, 0>(v[x][0][y], v[x][1][y], af[0][0], af[0][1]);
                two_keys_finite<FMT, 0>(v[x][2][y], v[x][3][y], af[0][2], af[0][3]);
                two_keys_finite<FMT, 2>(v[x][0][y], v[x][1][y], af[1][0], af[1][1]);
                two_keys_finite<FMT, 2>(v[x][2][y], v[x][3][y], af[1][2], af[1][3]);
              } else {
                two_keys<FMT, 0>(v[x][0][y], v[x][1][y], af[0][0], af[0][1]);
                two_keys<FMT, 0>(v[x][2][y], v[x][3][y], af[0][2], af[0][3]);
                two_keys<FMT, 2>(v[x][0][y], v[x][1][y], af[1][0], af[1][1]);
                two_keys<FMT, 2>(v[x][2][y], v[x][3][y], af[1][2], af[1][3]);
              }
#pragma unroll
              for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma(o[n][x * 8 + y * 2 + z], af[z], p[n][0], p[n][1]);
            }
        };
        if (FMT == MOE_DT_E4M3 && partly) values(std::true_type{});
        else values(std::false_type{});
      }
      // ---- the tile that takes this one's place: its scales by each warp, its codes by the last that is done
      const int next = i + kStages;
      if (next < tiles) {
        if (next % batch == 0) look_up(next);
        __syncwarp();
        ask_scales(next, st_no);
        int before = 0;
        if (lane == 0)
          asm volatile("atom.acq_rel.cta.shared::cta.add.s32 %0, [%1], 1;" : "=r"(before) : "r"(smem_u32(s_done + st_no)) : "memory");
        if (__shfl_sync(kAll, before, 0) == W - 1) {
          if (lane == 0) s_done[st_no] = 0;
          ask_codes(next, st_no);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
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
    float* const part = reinterpret_cast<float*>(a.ws + kWsHead) +
                        ((size_t)blockIdx.x * 2 + ((int)blockIdx.x == c0 ? 1 : 0)) * C::kPartFloats;
    const auto put_lse = [&](int r, float mm, float sum) {
      if (a.lse) {
        const int R = r0 + r, tok = quotient(R, G);
        a.lse[(int64_t)(w.s.q0 + tok) * a.Hq + h * G + R - tok * G] = lse_of(mm, sum);
      }
    };
    const auto row_at = [&](int r) {
      const int R = r0 + r, tok = quotient(R, G);
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
        out_factors(mm, mmv, sum, s_rf[tid], s_f[tid]);
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
        put(ga, row_at(r) + col * 4, times(v, s_rf[r], s_f[r]));
      } else {
        __stcg(reinterpret_cast<float4*>(part) + e, v);
      }
    }
    if (parts == 1) continue;

    // ---- an item of several CTAs: the last to arrive joins its parts
    __syncthreads();
    if (tid == 0) {  // (what the other threads wrote is ordered by the barrier)
      unsigned* counter = reinterpret_cast<unsigned*>(a.ws + 16) + c0;
      __threadfence();
      sh.last = atomicInc(counter, (unsigned)parts - 1) == (unsigned)parts - 1;  // wraps to 0 behind the last
      __threadfence();
    }
    __syncthreads();
    if (!sh.last) continue;
    const float* const part0 = reinterpret_cast<const float*>(a.ws + kWsHead);
    const auto part_of = [&](int p) { return part0 + ((size_t)(c0 + p) * 2 + (p == 0 ? 1 : 0)) * C::kPartFloats; };
    float* const wgt = reinterpret_cast<float*>(smem);  // [part][nr]
    constexpr int kHeld = kRows / W;  // a warp takes every W-th row, a lane a part
    float pm[kHeld], pv[kHeld], pl[kHeld], mm[kHeld], mmv[kHeld], sum[kHeld];
    const auto ask_rows = [&](int p) {
#pragma unroll
      for (int y = 0; y < kHeld; ++y) {
        pm[y] = pv[y] = kLow, pl[y] = 0.0f;
        const int r = y * W + warp;
        if (p < parts && r < nr) {
          const float* q = part_of(p) + kPartMax + r;
          pm[y] = __ldcg(q), pv[y] = __ldcg(q + 32), pl[y] = __ldcg(q + 64);
        }
      }
    };
#pragma unroll
    for (int y = 0; y < kHeld; ++y) mm[y] = mmv[y] = kLow, sum[y] = 0.0f;
#pragma unroll 1
    for (int p = lane; p < parts + lane; p += 32) {  // (every lane as often)
      ask_rows(p);
#pragma unroll
      for (int y = 0; y < kHeld; ++y) mm[y] = fmaxf(mm[y], pm[y]), mmv[y] = fmaxf(mmv[y], pv[y]);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
#pragma unroll
      for (int y = 0; y < kHeld; ++y) {
        mm[y] = fmaxf(mm[y], __shfl_xor_sync(kAll, mm[y], x));
        mmv[y] = fmaxf(mmv[y], __shfl_xor_sync(kAll, mmv[y], x));
      }
#pragma unroll 1
    for (int p = lane; p < parts + lane; p += 32) {
      if (parts > 32) ask_rows(p);
#pragma unroll
      for (int y = 0; y < kHeld; ++y) {
        sum[y] += pl[y] * ex2(pm[y] - mm[y]);
        if (p < parts && y * W + warp < nr) wgt[p * nr + y * W + warp] = ex2(pv[y] - mmv[y]);
      }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
#pragma unroll
      for (int y = 0; y < kHeld; ++y) sum[y] += __shfl_xor_sync(kAll, sum[y], x);
    if (lane == 0) {
#pragma unroll
      for (int y = 0; y < kHeld; ++y)
        if (y * W + warp < nr) {
          out_factors(mm[y], mmv[y], sum[y], s_rf[y * W + warp], s_f[y * W + warp]);
          put_lse(y * W + warp, mm[y], sum[y]);
        }
    }
    __syncthreads();
    const int n = nr * (D / 4);  // vectors of 4 columns
    int teams = 1;               // teams of threads share the parts where there are few
    while (teams * 2 * n <= kThreads && teams * 2 <= parts) teams *= 2;
    const int width = kThreads / teams, team = tid / width;
    const auto load = [&](int p, int e) { return __ldcg(reinterpret_cast<const float4*>(part_of(p)) + e); };
    const auto finish = [&](int e, float4 v) {
      const int r = e / (D / 4), col = e - r * (D / 4);
      put(ga, row_at(r) + col * 4, times(v, s_rf[r], s_f[r]));
    };
    constexpr int kAhead = 8;  // parts that are asked for together
    if (n <= width) {
      float4* const red = reinterpret_cast<float4*>(smem + C::kRing - kThreads * 16);
      const int e = tid - team * width, r = e / (D / 4);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (e < n) {
#pragma unroll 8
        for (int p = team; p < parts; p += teams) fma4(v, wgt[p * nr + r], load(p, e));
      }
      if (teams > 1) {
        red[tid] = v;
        __syncthreads();
        if (team == 0)
          for (int x = 1; x < teams; ++x) fma4(v, 1.0f, red[tid + x * width]);
      }
      if (team == 0 && e < n) finish(e, v);
    } else {
      constexpr int kB = 2;  // vectors of a thread
      for (int e0 = tid; e0 < n; e0 += kB * kThreads) {
        float4 v[kB];
        int row[kB];
#pragma unroll
        for (int x = 0; x < kB; ++x) v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f), row[x] = min(e0 + x * kThreads, n - 1) / (D / 4);
#pragma unroll 1
        for (int p0 = 0; p0 < parts; p0 += kAhead) {
          float4 in[kAhead][kB];
#pragma unroll
          for (int y = 0; y < kAhead; ++y)
#pragma unroll
            for (int x = 0; x < kB; ++x) in[y][x] = load(min(p0 + y, parts - 1), min(e0 + x * kThreads, n - 1));
#pragma unroll
          for (int y = 0; y < kAhead; ++y)
#pragma unroll
            for (int x = 0; x < kB; ++x)
              if (p0 + y < parts) fma4(v[x], wgt[(p0 + y) * nr + row[x]], in[y][x]);
        }
#pragma unroll
        for (int x = 0; x < kB; ++x)
          if (e0 + x * kThreads < n) finish(e0 + x * kThreads, v[x]);
      }
    }
  }
  if (sh.abort) {  // copies may be in flight still
    const long long t0 = clock64();
    while (clock64() - t0 < kWaitCycles / 8) {
    }
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// a cache's codes as [page][head][row][D]: boxes of `rows` rows of one head of one page, up to 128 columns
bool make_map(CUtensorMap* map, const moe_kv_desc& kv, const void* cache, int64_t row, int64_t head, int64_t page, int rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const auto bytes = [&](int64_t stride) { return (cuuint64_t)(stride ? stride : kv.D); };  // 0: one entry
  const cuuint64_t dims[4] = {(cuuint64_t)kv.D, (cuuint64_t)kv.page_size, (cuuint64_t)kv.Hkv, (cuuint64_t)kv.num_pages};
  const cuuint64_t strides[3] = {bytes(row), bytes(head), bytes(page)};
  const cuuint32_t box[4] = {(cuuint32_t)std::min(kv.D, 128), (cuuint32_t)rows, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(cache), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, kv.D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  const moe_kv_desc& kv = a.a.kv;
  CUtensorMap km, vm;
  const int rows = std::min(C::kTile, kv.page_size & -kv.page_size);
  if (!make_map(&km, kv, a.a.k_cache, kv.k_row_stride, kv.k_head_stride, kv.k_page_stride, rows) ||
      !make_map(&vm, kv, a.a.v_cache, kv.v_row_stride, kv.v_head_stride, kv.v_page_stride, rows))
    return cudaErrorInvalidValue;
  note_launch();
  return launch_overlapping(kern, dim3((unsigned)std::min(2 * num_sms(), kMaxCtas)), 32 * C::W, C::kSmem, 1, s, a, km, vm);
}
template <int D, int FMT>
cudaError_t launch_rows(const AttnQ8Args& g, cudaStream_t s) {
  // Rows of an item: those of a sequence of the mean number of new tokens.  A longer one has several items and reads its
  // keys as often, a shorter one leaves rows empty.  In us with 8 / 16 / 32 rows, 16 sequences of 4096 keys but for the last:
  //   rows of each       8               16              24              32              48              64
  //   D = 64, 8 heads    26 / 30 / 42    42 / 30 / 43    57 / 49 / 44    73 / 50 / 44    103 / 68 / 76   133 / 87 / 77
  //   D = 128, 4 heads   21 / 25 / 36    31 / 28 / 38    42 / 41 / 41    52 / 42 / 42    71 / 56 / 65    92 / 71 / 66
  //   D = 256, 2 heads   22 / 26         29 / 31         38 / 38         47 / 39         64 / 50         83 / 61
  //   2 of 65536, 128    39 / 45 / 65    50 / 52 / 73    72 / 69 / 78    88 / 71 / 83    126 / 99 / 117  163 / 125 / 118
  // Windows of 1 to 4 tokens of 5 heads of 64, whose mean are 15 rows: 42 / 35 / 44.  So 16 rows would be as good or better
  // than 32 up to 48 rows of 128 columns and from 33 to 48 of 64.
  const int64_t mean = (g.a.T + (int64_t)g.a.kv.n_seqs - 1) / g.a.kv.n_seqs, want = g.a.Hq / g.a.kv.Hkv * mean;
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
    if (v % 16 || v >= (int64_t)1 << 40) return false;  // (what a tensor map takes)
  // a stride of 0 over several entries (one key for all heads, say) is not one either
  const bool repeats = (kv.page_size > 1 && !(kv.k_row_stride && kv.v_row_stride)) ||
                       (kv.Hkv > 1 && !(kv.k_head_stride && kv.v_head_stride)) ||
                       (kv.num_pages > 1 && !(kv.k_page_stride && kv.v_page_stride));
  return !repeats && (kv.D == 64 || kv.D == 128 || kv.D == 256) && kv.page_size % 16 == 0 &&
         reinterpret_cast<uintptr_t>(g.a.k_cache) % 16 == 0 && reinterpret_cast<uintptr_t>(g.a.v_cache) % 16 == 0;
}

bool attn_q8_fits(const AttnQ8Args& g) {  // units are 32-bit numbers
  const moe_kv_desc& kv = g.a.kv;
  const int64_t items = ((int64_t)g.a.T * g.G / 8 + kv.n_seqs) * kv.Hkv;
  return items * ((int64_t)kv.max_pages * kv.page_size / 64 + 2 + kOver) < (int64_t)1 << 31;
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
