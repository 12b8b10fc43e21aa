// Attention of a chunk of new tokens over a paged key/value cache, on the
// tensor cores (tcgen05), for single tokens, verify windows and prompt chunks.
//
//   a_j = scale * q . k_j,   out = sum_j 2^(c a_j - m) v_j / sum_j 2^(c a_j - m)
//
// in one pass over the keys with a running reference m and sum (c = log2 e).
//
// Rows.  The query heads that share a key/value head are rows of the same
// tile: row R of a sequence is (token R / G, head R % G), so a single token
// of G heads already fills G rows and every key is read once per key/value
// head.  A work item is (sequence, key/value head, up to 256 rows) over its
// visible range of keys, cut into tiles of kN keys.
//
// Work split.  Each CTA (one per SM) finds its share of the items' key tiles
// from cu_q and kv_len in a short prologue: no planning launch, no host
// knowledge of the lengths.  Items stay whole where cutting them costs more
// than uneven work does; else equal numbers of CTAs share each item, or all
// tiles, laid end to end, are divided evenly whatever the lengths (see plan).
// A cut item leaves partial sums in the workspace; when all of them are there,
// its CTAs join a slice of its rows each, in a fixed order, so results do not
// depend on timing.
//
// What it measured: 2 prompts of up to 4096 new tokens over up to 16384 keys
// (32 heads over 4 of 128) 642 us, 1640 TFLOP/s, bound by the chain of the
// softmax and the products that feed it; 48 tokens over up to 8192 keys 76 us,
// 5.4 TB/s (6.6 to 6.9 where the lengths are equal); one token over 777 keys
// 11.3 us, latency.
//
// Inside a CTA (warp roles): one warp feeds a ring of key and value tiles by
// TMA through the page table, one issues the MMAs, two gather the query rows,
// and two groups of four warps run the softmax, each on its own score buffer
// in tensor memory, thread = row.  Score tile u uses buffer u % 2:
//   items of more than 128 rows: u = 2 * tile + half, each half a row tile of
//     its own (both read the same keys);
//   smaller items: u = tile, the two groups take alternate key tiles with
//     sums of their own and are joined at the end.
// The issue order S(0) S(1) | P(u)V, S(u + 2) | keeps one group's softmax
// beside the other's products.  P replaces its scores in tensor memory as
// 16-bit numbers (one rounding; sums are taken of the unrounded values) and
// is the A operand of P V; V is read as it lies in the cache (MN-major).
//
// The output accumulator is rescaled only when a row's maximum has grown by
// more than 2^8 over the reference: weights stay below 2^8 times the
// reference's, in range for fp16 and bf16, and most tiles skip the pass over
// the accumulator.
//
// Every wait is bounded: after about a second a role records
// MOE_ERR_DEVICE_TIMEOUT, and all roles run to the end without waiting.
#include <algorithm>
#include <cmath>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_kv.cuh"
#include "moe_per_device.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr long long kWaitCycles = 2000000000ll;  // ~1 s at 2 GHz
constexpr int kMaxCtas = 160;                    // the workspace holds the partial sums of this many
constexpr size_t kWsHead = 1024;                 // status (16 bytes), a counter per CTA
static_assert(kWsHead >= 16 + 4 * kMaxCtas, "counters");
// Units of work: a key tile counts 1, an item kItemUnits more (loading its
// queries, filling the pipeline, writing its rows).  3 lies between what was
// measured on an earlier form of this kernel: with 0, 2 and 4 units an
// 8192-token prompt (32 heads over 4, 128 wide) took 549, 422 and 402 us, 48
// decoded tokens over up to 8192 keys 82, 77 and 78 us.  (Fewer CTAs of 2 or 4
// units at least, where the work does not fill the SMs, were slower: one token
// over 777 keys 12 us, 14 and 19.)
constexpr int kItemUnits = 3;
constexpr float kGrow = 8.0f;                    // log2 of the growth that forces a rescale
// log2 of the reference's weight in 16-bit weights: up to 2^15 in fp16, whose normal numbers then reach down to 2^-21 of
// the reference (2^-14 without).  Below them a weight is off by up to 2^-32 of the reference.
template <bool BF16>
constexpr float kLiftOf = BF16 ? 0.0f : 7.0f;

template <int D_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int kN = D == 256 ? 64 : 128;         // keys per tile
  static constexpr int kGroups = D == 256 ? 1 : 2;       // softmax groups of four warps
  static constexpr int kRows = 128 * kGroups;            // rows per item
  static constexpr int kSub = D / 64;                    // 128-byte wide sub-tiles of a row
  static constexpr int kSlot = kN * D * 2;               // one key or value tile
  static constexpr int kQ = 128 * D * 2;                 // one row tile of q
  static constexpr int kStages = (229376 - kGroups * kQ) / kSlot;
  static constexpr int kThreads = 128 * kGroups + 128;
  static constexpr int kSmemQ = 0;
  static constexpr int kSmemRing = kGroups * kQ;
  static constexpr int kSmemMisc = kSmemRing + kStages * kSlot;
  static constexpr int kBars = 8 * (2 * kStages + 11);    // barriers of a pass
  static constexpr int kSmemStart = kSmemMisc + 2 * kBars;  // after those of two passes: the prologue's results
  static constexpr int kSmemXch = kSmemMisc + 1024;
  static constexpr int kSmem = kSmemXch + 2 * 128 * 8;   // per group and row: maximum and sum, for joining the groups
  static constexpr size_t kPartFloats = (size_t)kRows * (D + 2);  // m, sum and accumulator of an item's rows
  static constexpr uint32_t kColO = 0, kColS = 256;      // tensor memory columns: O per group, two score buffers
};
static_assert(Cfg<64>::kBars >= Cfg<128>::kBars && Cfg<64>::kBars >= Cfg<256>::kBars, "barriers");
static_assert(Cfg<128>::kSmem <= 232448 && Cfg<64>::kSmem <= 232448 && Cfg<256>::kSmem <= 232448, "shared memory");

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t bar, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t p, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// one K step of 16: A and B from shared memory / A from tensor memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((int)acc));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"((int)acc));
}
// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// 32 columns of the warp's 32 lanes, one lane (row) per thread
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ uint64_t f2(float x, float y) {
  return (uint64_t)__float_as_uint(x) | ((uint64_t)__float_as_uint(y) << 32);
}
__device__ __forceinline__ float f2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ float ex2(float x) {  // 2^x, within 2 ulp; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's results from its sum of weights, 2^m of them in all: 0 where it sees no key.  A sum that is no number (a NaN or
// an overflow in its scores) stays one.
__device__ __forceinline__ float inverse_of(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
__device__ __forceinline__ float lse_of(float m, float sum) {
  return sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945309f;
}

__device__ __forceinline__ void store32(void* p, const uint32_t* v) {  // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Shared-memory matrix descriptors, 128-byte swizzle; only the start address
// (bits 0-13, in 16 bytes) varies, so a step is an addition to the low word.
// K-major: 8-row groups 1024 bytes apart, K advances by 32 bytes per step of
// 16 inside the 128.  MN-major: 64 columns (128 bytes) of one K row per line,
// 8-row groups 1024 bytes apart along K, the next 64 columns `next` bytes on.
constexpr uint32_t kDescHi = (uint32_t)(1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr & 0x3FFFF) >> 4) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr, uint32_t next) {
  return ((addr & 0x3FFFF) >> 4) | (next >> 4) << 16;
}
// kind::f16, fp32 accumulation, M = 128
__host__ __device__ constexpr uint32_t idesc(bool bf16, int N, bool b_mn, bool neg_a) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (neg_a ? 1u << 13 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t)(N >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

// ---------------------------------------------------------------- work items
// One item: a row tile of a (sequence, key/value head) and its range of keys.
struct Item {
  int b, h, i;       // sequence, key/value head, row tile
  SeqInfo s;
  int tiles_q;       // row tiles of the sequence
  int r0, rows;      // first row, rows (1 .. kRows)
  int lo, hi;        // keys that some row sees
  int t0, tiles;     // first key tile, number of key tiles
  __device__ __forceinline__ int payload() const { return max(1, tiles); }  // an item without keys still writes its rows
  __device__ __forceinline__ int cost() const { return kItemUnits + payload(); }
};

template <int kN, int kRows>
__device__ __forceinline__ void item_range(const AttnArgs& a, int G, Item& it) {
  const int R = it.s.n * G;
  it.r0 = it.i * kRows;
  it.rows = min(kRows, R - it.r0);
  const int off = it.s.kv - it.s.n;
  it.hi = max(0, off + (it.r0 + it.rows - 1) / G + 1);
  it.lo = min(it.hi, window_lo(off + it.r0 / G + 1, a.window));
  it.t0 = it.lo / kN;
  it.tiles = it.hi > it.lo ? (it.hi + kN - 1) / kN - it.t0 : 0;
}

// The CTA's run of work: `left` units from unit `off` of the current item on
// (by_item: a unit is a whole item, off = 0).
struct Walk {
  Item it;
  int off;
  int left;
  bool by_item;
};

// An item whose units several CTAs share (this CTA holds at most two of them).
struct Cut {
  int c0, parts, slot0;  // first CTA, number of CTAs, the first one's slot (the others use slot 0)
  int rows, r0, q0, h;
  int arrived;           // all parts are there (written once, before the barrier behind which it is read)
};

// what the prologue leaves in shared memory for every role
struct Start {
  Item item;  // the CTA's first, and the unit it starts with
  int off;
  int first, left;  // units
  int per, extra;   // units per CTA of the call, and how many CTAs' worth of remainder (see share)
  int ctas;
  bool by_item;     // units are whole items (see plan)
  int c0, parts;    // equal numbers of CTAs for the items: the first CTA of this item, and how many take part (else 0)
  volatile int abort;
  volatile int again;  // some output was not finite: a second pass (see clean_values)
  uint32_t tmem;
  int n_cut;
  Cut cut[2];
};

// Keys that every row of an item sees; the others of the item's range some rows see and some do not.
struct Shared {
  int lo, hi;
};
__device__ __forceinline__ Shared shared_keys(const AttnArgs& a, int G, const Item& it) {
  return Shared{window_lo(it.hi, a.window), max(it.lo, it.s.kv - it.s.n + it.r0 / G + 1)};
}

static_assert(2 * Cfg<64>::kBars + sizeof(Start) <= 1024 && Cfg<64>::kBars % 8 == 0, "shared memory after the barriers");

__device__ __forceinline__ Walk walk_begin(const Start& st) {
  Walk w;
  w.it = st.item;
  w.off = st.off;
  w.left = st.left;
  w.by_item = st.by_item;
  return w;
}
// past the current item, if work is left
template <int kN, int kRows>
__device__ __forceinline__ void walk_next(const AttnArgs& a, int G, Walk& w, int done) {
  w.left -= done;
  if (w.left <= 0) return;
  w.off = 0;
  if (++w.it.i == w.it.tiles_q) {
    w.it.i = 0;
    if (++w.it.h == a.kv.Hkv) {
      w.it.h = 0;
      do {
        ++w.it.b;
        w.it.s = seq_info(a.kv, a.cu_q, a.kv_len, a.T, w.it.b);
      } while (w.it.s.n == 0 && w.it.b + 1 < a.kv.n_seqs);
      w.it.tiles_q = (w.it.s.n * G + kRows - 1) / kRows;
    }
  }
  item_range<kN, kRows>(a, G, w.it);
}
// What of the current item is this CTA's: `len` units, of which the payload
// [first, last) (none: the CTA's boundary fell into the item's overhead, and
// the item is the next CTA's), `tiles` key tiles of it.
struct Seg {
  int len, first, last, tiles;
};
__device__ __forceinline__ Seg walk_seg(const Walk& w) {
  Seg s;
  s.len = w.by_item ? 1 : min(w.it.cost() - w.off, w.left);
  s.first = max(w.off - kItemUnits, 0);
  s.last = w.by_item ? w.it.payload() : max(w.off + s.len - kItemUnits, 0);
  s.tiles = w.it.tiles ? s.last - s.first : 0;
  return s;
}

// a / b for 0 <= a < 2^16, 0 < b <= kMaxCtas: the quotient of a + 1/2 lies at
// least 1 / (2 b) from a whole number, far more than its error
__device__ __forceinline__ int small_div(int a, int b) { return (int)__fdividef((float)a + 0.5f, (float)b); }

// How a call's work is divided: whole items, as even in number as they go; or,
// where items are few, an equal number of CTAs for each; or even shares of all
// units.  Even shares finish together, but an item that is cut costs its parts'
// way through the workspace and their join, and the more, the more of the CTAs
// hold parts of two items.  In units, with X = rows * D / (16 threads) for what
// a thread of the softmax groups writes and reads of a part, a CTA is done after
//   whole items       most * ceil(items / ctas)
//   equal numbers     most / (ctas / items)  +  7 + X / 5
//   even shares       units / ctas  +  7 + X / 5  +  (12 + X) / max(2, ctas / items)
// and the least is taken; the constants are fits to 800 measured shapes.  With
// 152 CTAs, in us:                          whole items  equal numbers  even shares
//   64 items of   8 rows of 128,  512 keys         11.2           12.7         14.1
//   64 items of   8 rows of 128, 2048 keys         23.3           21.9         24.6
//   32 items of   8 rows of 128, 8192 keys         67.8           32.4         32.9
//   64 items of 128 rows of 128, 1024 keys         17.4           18.8         26.2
//   32 items of 128 rows of 256, 4096 keys         65.5           39.2         48.2
//  100 items of 128 rows of 256, 1024 keys         28.9              -         53.3
//  200 items of   8 rows of  64,  512 keys         15.8              -         21.7
struct Plan {
  bool by_item;
  int each;  // CTAs of an item (by_item; 0: whole items, any number to a CTA)
  int units, ctas;
};
template <int D, int kRows>
__device__ __forceinline__ Plan plan(int units, int items, int most, int rows) {  // most: units of the largest item
  // (fp32 will do: every CTA comes to the same plan, and any plan is right.)
  const int grid = gridDim.x;
  const float even = __fdividef((float)units, (float)grid), ratio = __fdividef((float)grid, (float)items);
  const float x = (float)(min(rows, kRows) * D) * (1.0f / (16 * kRows));
  const float joined = 7.0f + 0.2f * x;
  const int each = max(1, (int)(ratio + 0.01f));
  const float whole = (float)most * ceilf(__fdividef((float)items, (float)grid));
  const float equal = each > 1 ? __fdividef((float)most, (float)each) + joined : INFINITY;
  const float shares = even + joined + __fdividef(12.0f + x, fmaxf(ratio, 2.0f));
  if (items && whole <= fminf(equal, shares)) return Plan{true, 0, items, min(grid, items)};
  if (items && equal <= shares) return Plan{true, each, items, items * each};
  return Plan{false, 0, units, max(1, min(grid, units))};
}

// units before CTA c
// (A call has fewer than 2^31 units: attn_units_fit.)
__device__ __forceinline__ int share(const Start& st, int c) { return c * st.per + small_div(c * st.extra, st.ctas); }
// the CTA that holds unit g: a guess, put right
__device__ __forceinline__ int owner(const Start& st, int g) {
  int c = min((int)(((float)g + 0.5f) / ((float)st.per + (float)st.extra / (float)st.ctas)), st.ctas - 1);
  while (share(st, c) > g) --c;
  while (c + 1 < st.ctas && share(st, c + 1) <= g) ++c;
  return c;
}

struct Wait {
  Start* st;
  int* status;
  // false: given up here or by another role
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(bar, parity)) {
      if (st->abort) return false;
      if (clock64() - t0 > kWaitCycles) {
        st->abort = 1;
        set_status(status, MOE_ERR_DEVICE_TIMEOUT);
        return false;
      }
    }
    return true;
  }
};

// every lane of a (converged) warp waits; the warp is converged afterwards.  A
// wait that was given up is not told: the softmax groups run on, so that all
// of them reach the same barriers, and the result is void (status word).
__device__ __forceinline__ void warp_wait(const Wait& w, uint32_t bar, uint32_t parity) {
  w(bar, parity);
  __syncwarp();
}

__device__ __forceinline__ void fma4(float4& acc, float f, float4 v) {
  acc.x = fmaf(f, v.x, acc.x);
  acc.y = fmaf(f, v.y, acc.y);
  acc.z = fmaf(f, v.z, acc.z);
  acc.w = fmaf(f, v.w, acc.w);
}
// release / acquire at GPU scope; the CTA's other threads are ordered by the barriers around them
__device__ __forceinline__ void count_up(unsigned* counter, int wrap) {
  asm volatile("fence.acq_rel.gpu;\n red.relaxed.gpu.global.inc.u32 [%0], %1;" ::"l"(counter), "r"(wrap) : "memory");
}
__device__ __forceinline__ void count_gone(unsigned* counter, int wrap) {  // what was read has been used already
  asm volatile("red.relaxed.gpu.global.inc.u32 [%0], %1;" ::"l"(counter), "r"(wrap) : "memory");
}
__device__ __forceinline__ unsigned count_read(const unsigned* counter) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
  return v;
}

// A part's accumulator, in vectors of 4 columns: the rows of a vector next to
// each other, so that a warp's stores (thread = row) and the loads of a slice
// of rows both take whole sectors; the vectors of a row next to each other
// where the CTAs join one row each and a part has few (one token of 8 heads of
// 256 over 32768 keys: 26 against 29 us; a prompt of 78 tokens of 8 heads of
// 256 over 7275 keys: 31 against 25).
__device__ __forceinline__ bool part_by_row(int rows, int parts) { return rows <= min(parts, 32); }

// Joins one item's parts.  Every one of its CTAs takes a slice of the rows,
// once all parts have arrived; the softmax threads of the CTA take part.
//   M = max_p m_p,  L = sum_p 2^(m_p - M) l_p,  out = sum_p 2^(m_p - M) o_p / L
// in the order of the parts.  (One CTA joining all rows of an item took up to
// 250 us for 128 rows in 30 parts; in slices it is bound by the L2 reads.)
template <int D, bool BF16>
__device__ __forceinline__ void join_parts(const AttnArgs& a, int G, Start& st, Cut& cut, const float* part0,
                                           unsigned* counters, uint8_t* smem) {
  using C = Cfg<D>;
  constexpr int kThreads = 128 * C::kGroups, kVecs = D / 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int np = cut.parts;
  // One counter per item, named by its first CTA: up to np as the parts are
  // written, up to 2 np as the CTAs have read them, where it wraps to 0.
  unsigned* counter = counters + cut.c0;
  if (tid == 0) {
    const long long t0 = clock64();
    while (count_read(counter) < (unsigned)np && !st.abort) {
      if (clock64() - t0 > kWaitCycles) {
        st.abort = 1;
        set_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
      }
    }
    cut.arrived = count_read(counter) >= (unsigned)np;
  }
  named_sync(4, kThreads);
  // Given up: the call is void.  Every thread reads the flag of this item, which no later item's wait writes, so all of
  // them leave here or none does, and all meet the same barriers afterwards.
  if (!cut.arrived) return;
  const int per = (cut.rows + np - 1) / np, lo = ((int)blockIdx.x - cut.c0) * per;
  const int nr = min(per, cut.rows - lo);
  const auto part = [&](int p) { return part0 + ((size_t)(cut.c0 + p) * 2 + (p == 0 ? cut.slot0 : 0)) * C::kPartFloats; };
  float* wgt = reinterpret_cast<float*>(smem);               // [np][per] weights over L: at most rows + np of them
  float4* red = reinterpret_cast<float4*>(smem + 4096);      // [thread] partial sums
  const auto finish = [&](int row, float M, float L) {
    if (a.lse) {
      const int R = cut.r0 + lo + row, tok = R / G;
      a.lse[(int64_t)(cut.q0 + tok) * a.Hq + cut.h * G + (R - tok * G)] =
          lse_of(M, L);
    }
  };
  const int n = nr > 0 ? nr * kVecs : 0;  // vectors of 4 columns
  int teams = 1;                          // teams of threads share the parts where there are few vectors
  while (n && teams * 2 * n <= kThreads && teams * 2 <= np) teams *= 2;
  const int width = kThreads / teams, team = tid / width;
  const bool single = n <= width;  // one vector per thread
  const bool by_row = part_by_row(cut.rows, np);
  const int cs = by_row ? 1 : cut.rows, rs = by_row ? kVecs : 1;  // steps of a vector's column and row
  const auto load = [&](const float* src, int row, int v) {
    return __ldcg(reinterpret_cast<const float4*>(src) + v * cs + (lo + row) * rs);
  };
  // one vector per thread: the first parts are asked for before the weights are known
  constexpr int kAhead = 8;
  float4 ahead[kAhead];
  const int my = tid % width, my_v = small_div(my, max(nr, 1)), my_row = my - my_v * nr;
  if (single && my < n) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (team + i * teams < np) ahead[i] = load(part(team + i * teams) + 2 * C::kRows, my_row, my_v);
  }
  if (np <= 8) {  // many rows each: a thread per row, its loads together
    for (int row = tid; row < nr; row += kThreads) {
      float m[8], l[8], M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float2 ml = p < np ? __ldcg(reinterpret_cast<const float2*>(part(p)) + lo + row) : make_float2(-INFINITY, 0.0f);
        m[p] = ml.x;
        l[p] = ml.y;
        M = fmaxf(M, m[p]);
      }
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        m[p] = m[p] == -INFINITY ? 0.0f : ex2(m[p] - M);
        L += m[p] * l[p];
      }
      const float il = inverse_of(L);
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p < np) wgt[p * per + row] = m[p] * il;
      finish(row, M, L);
    }
  } else {  // few rows each: a warp per row, a lane per part
    constexpr int kPer = (kMaxCtas + 31) / 32;
    for (int row = warp; row < nr; row += kThreads / 32) {
      float m[kPer], M = -INFINITY, L = 0.0f;
      float l[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int p = i * 32 + lane;
        const float2 ml = p < np ? __ldcg(reinterpret_cast<const float2*>(part(p)) + lo + row) : make_float2(-INFINITY, 0.0f);
        m[i] = ml.x;
        l[i] = ml.y;
        M = fmaxf(M, m[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        m[i] = m[i] == -INFINITY ? 0.0f : ex2(m[i] - M);
        L += m[i] * l[i];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(kAll, L, o);
      const float il = inverse_of(L);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int p = i * 32 + lane;
        if (p < np) wgt[p * per + row] = m[i] * il;
      }
      if (lane == 0) finish(row, M, L);
    }
  }
  named_sync(4, kThreads);
  if (nr > 0) {  // uniform over the CTA
    const auto put = [&](int row, int col, float4 v) {
      const int R = cut.r0 + lo + row, tok = R / G;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (int64_t)(cut.q0 + tok) * a.o_stride +
                                (int64_t)(cut.h * G + R - tok * G) * a.o_head_stride + 4 * col) =
          make_uint2(pack16<BF16>(v.x, v.y), pack16<BF16>(v.z, v.w));
    };
    if (single) {
      if (my < n) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (team + i * teams < np) fma4(acc, wgt[(team + i * teams) * per + my_row], ahead[i]);
#pragma unroll 8
        for (int p = team + kAhead * teams; p < np; p += teams)
          fma4(acc, wgt[p * per + my_row], load(part(p) + 2 * C::kRows, my_row, my_v));
        if (teams > 1) red[tid] = acc;
        else put(my_row, my_v, acc);
      }
    } else {  // several vectors of a thread in flight
      constexpr int kB = 4;
      for (int e0 = tid; e0 < n; e0 += kB * width) {
        float4 acc[kB];
        int row[kB], c[kB];
#pragma unroll
        for (int i = 0; i < kB; ++i) {
          const int e = min(e0 + i * width, n - 1);  // the last vector again where there is none
          acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          c[i] = small_div(e, nr);
          row[i] = e - c[i] * nr;
        }
#pragma unroll (C::kGroups == 1 ? 4 : 2)  // a group of threads less: more loads of each in flight
        for (int p = 0; p < np; ++p) {
          const float* src = part(p) + 2 * C::kRows;
#pragma unroll
          for (int i = 0; i < kB; ++i) fma4(acc[i], wgt[p * per + row[i]], load(src, row[i], c[i]));
        }
#pragma unroll
        for (int i = 0; i < kB; ++i)
          if (e0 + i * width < n) put(row[i], c[i], acc[i]);
      }
    }
    if (teams > 1) {
      named_sync(4, kThreads);
      if (tid < n) {
        float4 acc = red[tid];
        for (int t = 1; t < teams; ++t) {
          const float4 v = red[t * width + tid];
          acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
        put(my_row, my_v, acc);
      }
    }
  }
  named_sync(4, kThreads);  // every read of the parts and of shared memory is done
  if (tid == 0) count_gone(counter, np * 2 - 1);
}

// All ones in each half of a word whose 16-bit number is not finite.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t kExp = BF16 ? 0x7f807f80u : 0x7c007c00u;
  return __vcmpeq2(w & kExp, kExp);
}
// Eight numbers times 0, added up: 0 (false) where all are finite, else NaN.
template <bool BF16>
__device__ __forceinline__ bool times_zero(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w[i]), "r"(0u));
    else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w[i]), "r"(0u));
  }
  return (sum & 0x7fff7fffu) != 0;
}
// Values that some row of an item multiplies by 0, because it does not see their key, have to be finite: 0 times infinity
// is NaN.  The issuing thread clears what lies outside the item's range of keys.  Keys that some rows of an item see and
// some do not (later tokens of the chunk, the far end of a window) are looked at only when a row's output turned out not
// to be finite although its sum is: the CTA then does its work again, and in that pass the 128 threads of a softmax group
// look through the values of the tile's rows [s0, e) and [b, s1), which are those keys, before they hand over the tile's
// weights.  What is not finite is cleared, and the rows that do see it get it back with their results (see add_cleared).
// With two row tiles both groups do so, each before its own product, on the same tile: they clear the same elements.
// (Looking in the first pass made items of few tiles 5 to 15% longer: by the softmax groups, or by the warps that gather
// the query rows.)
template <int D, bool BF16>
__device__ __forceinline__ void clean_values(uint32_t tile, int s0, int e, int b, int s1, int r) {
  constexpr int kN = Cfg<D>::kN, kChunks = D / 8;
  const int n0 = (e - s0) * kChunks, n = n0 + (s1 - b) * kChunks;
#pragma unroll 1
  for (int i = r; i < n; i += 128) {
    const int row = (i < n0 ? s0 : b - (e - s0)) + i / kChunks, ch = i % kChunks;
    const uint32_t p = tile + (ch / 8) * (kN * 128) + row * 128 + (ch % 8) * 16;
    const auto keep = [](uint32_t w) { return w & ~not_finite<BF16>(w); };
    const uint4 v = lds16(p);
    if (times_zero<BF16>(v)) sts16(p, make_uint4(keep(v.x), keep(v.y), keep(v.z), keep(v.w)));
  }
  fence_proxy();  // the products read shared memory by the async proxy
}
// Adds the values that clean_values takes out to the columns [col0, col1) of a row that sees the keys [j0, j1) of a
// segment: the infinity or NaN of the value, whatever the row's weight.  The row's result is in `out`, or where that is
// null in `part`, vectors of four columns `cs` vectors apart.
template <bool BF16>
__device__ __forceinline__ void add_cleared(const AttnArgs& a, int b, int h, int j0, int j1, Shared all, int col0, int col1,
                                            uint16_t* out, float* part, int cs) {
#pragma unroll 1
  for (int j = j0; j < j1; ++j) {
    if (j >= all.lo && j < all.hi) {
      j = all.hi - 1;
      continue;
    }
    const int page = __ldg(a.table + (int64_t)b * a.kv.table_stride + j / a.kv.page_size);
    if (page < 0 || page >= a.kv.num_pages) continue;
    const uint16_t* v = static_cast<const uint16_t*>(a.v_cache) + page * a.kv.v_page_stride +
                        (j % a.kv.page_size) * a.kv.v_row_stride + h * a.kv.v_head_stride;
#pragma unroll 1
    for (int c = col0; c < col1; ++c) {
      const uint32_t x = __ldg(v + c);
      if (!(not_finite<BF16>(x) & 1u)) continue;
      const float f = BF16 ? __uint_as_float(x << 16) : __half2float(__ushort_as_half((unsigned short)x));
      if (out) {
        const float o = BF16 ? __uint_as_float((uint32_t)out[c] << 16) : __half2float(__ushort_as_half(out[c]));
        out[c] = (uint16_t)pack16<BF16>(o + f, 0.0f);
      } else {
        part[(c / 4 * cs) * 4 + c % 4] += f;
      }
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
attn_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D>;
  constexpr int kN = C::kN, kRows = C::kRows, kGroups = C::kGroups, kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  if (base & 1023) {  // the swizzled tiles need it; no static shared memory comes before
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  uint32_t bars = base + C::kSmemMisc;
  const auto full = [&](int s) { return bars + 8 * s; };
  const auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  const auto drain = [&] { return bars + 8 * (2 * kStages); };
  const auto q_full = [&](int t) { return drain() + 8 + 8 * t; };    // row tile t of q is there
  const auto q_empty = [&](int t) { return drain() + 24 + 8 * t; };  // its last product is done
  const auto s_full = [&](int b) { return drain() + 40 + 8 * b; };   // scores of buffer b
  const auto p_full = [&](int b) { return drain() + 56 + 8 * b; };   // weights of buffer b
  const auto o_full = [&](int b) { return drain() + 72 + 8 * b; };   // buffer b's product with the values
  Start& st = *reinterpret_cast<Start*>(smem + C::kSmemStart);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarpLoad = 4 * kGroups, kWarpMma = kWarpLoad + 1, kWarpQ = kWarpLoad + 2;
  const int G = a.Hq / a.kv.Hkv;

  // ---- prologue: the call's work in units, and this CTA's share
  const auto init_barriers = [&] {
    for (int s = 0; s < kStages; ++s) {
      bar_init(full(s), 1);
      bar_init(empty(s), 1);
    }
    bar_init(drain(), 1);
    for (int b = 0; b < 2; ++b) {
      bar_init(q_full(b), 64);
      bar_init(q_empty(b), 1);
      bar_init(s_full(b), 1);
      bar_init(p_full(b), 4);
      bar_init(o_full(b), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  };
  if (warp == kWarpMma && lane == 0) {
    init_barriers();
    st.abort = 0;
    st.again = 0;
    st.n_cut = 0;
  }
  if (warp == kWarpMma) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&st.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // The units of 32 sequences, a lane per sequence (one of more than four row tiles is counted by the warp).
  struct Count {
    int units, items, most;  // most: units of the largest item
  };
  const auto count = [&](int b, SeqInfo& s) {
    Item it;
    s = SeqInfo{0, 0, 0, true};
    if (b < a.kv.n_seqs) s = seq_info(a.kv, a.cu_q, a.kv_len, a.T, b);
    if (!s.ok && blockIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    it.s = s;
    const int nt = (s.n * G + kRows - 1) / kRows;
    Count mine{0, nt * a.kv.Hkv, 0};
    if (nt <= 4) {
      for (it.i = 0; it.i < nt; ++it.i) {
        item_range<kN, kRows>(a, G, it);
        mine.units += it.cost();
        mine.most = max(mine.most, it.cost());
      }
    }
    for (unsigned many = __ballot_sync(kAll, nt > 4); many; many &= many - 1) {
      const int src = __ffs(many) - 1;
      Item x;
      x.s = SeqInfo{0, __shfl_sync(kAll, s.n, src), __shfl_sync(kAll, s.kv, src), true};
      const int nx = __shfl_sync(kAll, nt, src);
      int sum = 0, most = 0;
      for (x.i = lane; x.i < nx; x.i += 32) {
        item_range<kN, kRows>(a, G, x);
        sum += x.cost();
        most = max(most, x.cost());
      }
      sum = __reduce_add_sync(kAll, sum);
      most = __reduce_max_sync(kAll, most);
      if (lane == src) mine.units = sum, mine.most = most;
    }
    mine.units *= a.kv.Hkv;
    return mine;
  };
  // Whether sequences share rows of q, by the number of tokens that this lane's name.  Sequences follow one another in
  // cu_q, so only a cu_q out of order can make them overlap, and then their sum is no longer bounded by T, nor the
  // units by what the host allowed: nothing is computed.  (One of the sequences is reported in any case.)
  const auto overlap = [&](long long tokens) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tokens += __shfl_xor_sync(kAll, tokens, o);
    return tokens > a.T;
  };
  const auto scan = [&](auto v) {  // inclusive, over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const auto u = __shfl_up_sync(kAll, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  // warp 0: the CTA's units [g0, g1) start `rem` units into sequence it.b, of `mine` units in all
  const auto locate = [&](Item& it, const Plan& pl, int mine, int rem) {
    const int nt = it.tiles_q = (it.s.n * G + kRows - 1) / kRows;
    const int per = mine / a.kv.Hkv;
    it.h = rem / per;
    rem -= it.h * per;
    if (pl.by_item) {
      it.i = rem;
      item_range<kN, kRows>(a, G, it);
      int off = 0;
      if (lane == 0) {
        st.item = it;
        if (pl.each) {  // this CTA's part of the payload
          const int parts = min(pl.each, it.payload()), part = blockIdx.x - st.first * pl.each;
          const int q = it.payload() / parts, r = it.payload() - q * parts;
          const int first = part * q + small_div(part * r, parts), last = (part + 1) * q + small_div((part + 1) * r, parts);
          off = first ? kItemUnits + first : 0;
          st.c0 = st.first * pl.each;
          st.parts = parts;
          st.left = part < parts ? kItemUnits + last - off : 0;
        }
      }
      return off;
    }
    for (int i0 = 0; i0 < nt; i0 += 32) {
      it.i = i0 + lane;
      int units = 0;
      if (it.i < nt) {
        item_range<kN, kRows>(a, G, it);
        units = it.cost();
      }
      if (nt == 1) {  // a decode step
        if (lane == 0) st.item = it;
        return rem;
      }
      const int inc = scan(units);
      const unsigned hit = __ballot_sync(kAll, inc > rem);
      if (hit) {
        const int src = __ffs(hit) - 1;
        rem -= __shfl_sync(kAll, inc - units, src);
        if (lane == src) st.item = it;
        return rem;
      }
      rem -= __shfl_sync(kAll, inc, 31);
    }
    return rem;
  };
  const auto begin = [&](const Plan& pl, int& g0) {  // this CTA's share; false: none
    const int total = pl.units, n = pl.ctas, c = blockIdx.x;
    const bool work = c < n && total > 0;
    const int per = pl.each ? 0 : total / n, extra = total - per * n;
    g0 = !work ? 0 : pl.each ? small_div(c, pl.each) : c * per + small_div(c * extra, n);
    if (lane == 0) {
      st.off = 0;
      st.first = g0;
      st.left = work ? (c + 1) * per + small_div((c + 1) * extra, n) - g0 : 0;
      st.per = per;
      st.extra = extra;
      st.ctas = n;
      st.by_item = pl.by_item && !pl.each;
      st.parts = 0;
    }
    return work;
  };
  if (a.kv.n_seqs <= 32) {  // one warp's lanes hold all sequences
    if (warp == 0) {
      Item it;
      const Count my = count(lane, it.s);
      Plan pl = plan<D, kRows>(__reduce_add_sync(kAll, my.units), __reduce_add_sync(kAll, my.items),
                                     __reduce_max_sync(kAll, my.most), __reduce_max_sync(kAll, it.s.n) * G);
      if (__any_sync(kAll, !it.s.ok) && overlap(it.s.n)) pl = Plan{false, 0, 0, 1};
      const int mine = pl.by_item ? my.items : my.units, inc = scan(mine);
      int g0;
      if (begin(pl, g0)) {
        const int src = __ffs(__ballot_sync(kAll, inc > g0)) - 1;
        it.b = src;
        it.s = SeqInfo{__shfl_sync(kAll, it.s.q0, src), __shfl_sync(kAll, it.s.n, src), __shfl_sync(kAll, it.s.kv, src),
                       true};
        const int whole = __shfl_sync(kAll, mine, src), before = __shfl_sync(kAll, inc, src) - whole;
        const int off = locate(it, pl, whole, g0 - before);
        if (lane == 0) st.off = off;
      }
    }
  } else {
    // per sequence its units, its items; then per warp the largest item, the most tokens, whether one is bad; the ring is not in use yet
    int* units = reinterpret_cast<int*>(smem + C::kSmemRing);
    int *items = units + MOE_MAX_SEQS, *peaks = items + MOE_MAX_SEQS;
    static_assert(C::kStages * C::kSlot >= 4 * (2 * MOE_MAX_SEQS + 3 * C::kThreads / 32), "counts of the sequences");
    int most = 0, tokens = 0;
    bool bad = false;
    for (int b0 = warp * 32; b0 < a.kv.n_seqs; b0 += C::kThreads) {
      SeqInfo s;
      const Count my = count(b0 + lane, s);
      if (b0 + lane < a.kv.n_seqs) units[b0 + lane] = my.units, items[b0 + lane] = my.items;
      most = max(most, my.most);
      tokens = max(tokens, s.n);
      bad |= __any_sync(kAll, !s.ok);
    }
    most = __reduce_max_sync(kAll, most);
    tokens = __reduce_max_sync(kAll, tokens);
    if (lane == 0) peaks[3 * warp] = most, peaks[3 * warp + 1] = tokens, peaks[3 * warp + 2] = bad;
    __syncthreads();
    if (warp == 0) {
      int all_units = 0, all_items = 0;
      for (int b = lane; b < a.kv.n_seqs; b += 32) all_units += units[b], all_items += items[b];
      most = lane < C::kThreads / 32 ? peaks[3 * lane] : 0;
      tokens = lane < C::kThreads / 32 ? peaks[3 * lane + 1] : 0;
      bad = __any_sync(kAll, lane < C::kThreads / 32 && peaks[3 * lane + 2]);
      Plan pl = plan<D, kRows>(__reduce_add_sync(kAll, all_units), __reduce_add_sync(kAll, all_items),
                                     __reduce_max_sync(kAll, most), __reduce_max_sync(kAll, tokens) * G);
      if (bad) {
        long long all = 0;
        for (int b = lane; b < a.kv.n_seqs; b += 32) all += seq_info(a.kv, a.cu_q, a.kv_len, a.T, b).n;
        if (overlap(all)) pl = Plan{false, 0, 0, 1};
      }
      const int* cost = pl.by_item ? items : units;
      int g0;
      if (begin(pl, g0)) {
        int at = 0;  // units before the 32 sequences
        for (int b0 = 0; b0 < a.kv.n_seqs; b0 += 32) {
          const int b = b0 + lane;
          const int mine = b < a.kv.n_seqs ? cost[b] : 0, inc = scan(mine);
          const unsigned hit = __ballot_sync(kAll, at + inc > g0);
          if (hit) {
            const int src = __ffs(hit) - 1;
            Item it;
            it.b = b0 + src;
            it.s = seq_info(a.kv, a.cu_q, a.kv_len, a.T, it.b);
            const int whole = __shfl_sync(kAll, mine, src), before = at + __shfl_sync(kAll, inc, src) - whole;
            const int off = locate(it, pl, whole, g0 - before);
            if (lane == 0) st.off = off;
            break;
          }
          at += __shfl_sync(kAll, inc, 31);
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  fence_proxy();  // the prologue's writes to the ring come before the TMA's
  const uint32_t tmem = st.tmem;
  const Wait wait{&st, a.status};
  const float c2 = fmaxf(fabsf(a.scale) * 1.44269504088896341f, 1e-30f);  // log2 units; the sign is in the MMA

  // ---- softmax: thread = row
  const auto softmax = [&](auto pass) {
    constexpr bool kCareful = decltype(pass)::value;
    const int grp = warp >> 2, r = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
    const uint32_t o_addr = lanes + C::kColO + grp * D;
    uint32_t s_phase = 0, o_phase = 0;  // bit b: parity of buffer b's next scores / of its last product
    constexpr float kLift = kLiftOf<BF16>;
    float* const part0 = reinterpret_cast<float*>(a.ws + kWsHead);
    constexpr size_t kPartFloats = C::kPartFloats;
    float2* const xch = reinterpret_cast<float2*>(smem + C::kSmemXch);
    int g_seg = st.first;  // unit at which the segment starts
    int ring = 0;          // tiles that the segments before took from the ring (careful)
    // rows of out on 32-byte boundaries: whole sectors at a time
    const bool wide_out = ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)(a.o_stride * 2) | (uintptr_t)(a.o_head_stride * 2)) & 31) == 0;
    for (Walk w = walk_begin(st); w.left > 0;) {
      const Seg sg = walk_seg(w);
      if (sg.first == sg.last) {
        g_seg += sg.len;
        walk_next<kN, kRows>(a, G, w, sg.len);
        continue;
      }
      const int m = sg.tiles;
      const bool two = kGroups == 2 && w.it.rows > 128;
      const int U = two ? 2 * m : m;
      const int row = (two ? grp * 128 : 0) + r;  // row of the item
      const bool valid = row < w.it.rows;
      const bool busy = (row & ~31) < w.it.rows;  // some row of the warp exists
      const int R = w.it.r0 + row, tok = valid ? R / G : 0, g = valid ? R - tok * G : 0;
      const int pos = w.it.s.kv - w.it.s.n + tok;
      const int hi = pos + 1, lo = window_lo(hi, a.window);
      float ref = -INFINITY, sum = 0.0f;  // reference (raw score units) and sum of the row
      bool acc = false;                   // the accumulator holds something

      for (int u = kGroups == 2 ? grp : 0; u < U; u += kGroups) {
        const int buf = u & 1;
        warp_wait(wait, s_full(buf), s_phase >> buf & 1);
        s_phase ^= 1u << buf;
        fence_after();
        if (busy) {
          const uint32_t s_addr = lanes + C::kColS + buf * kN;
          uint32_t s[kN];
#pragma unroll
          for (int x = 0; x < kN / 32; ++x) tmem_ld32(s_addr + 32 * x, s + 32 * x);
          wait_ld();
          const int k0 = (w.it.t0 + sg.first + (two ? u >> 1 : u)) * kN;
          if (__any_sync(kAll, valid && (hi < k0 + kN || lo > k0))) {
            const int j1 = hi - k0, j0 = lo - k0;
#pragma unroll
            for (int j = 0; j < kN; ++j)
              if (j >= j1 || j < j0) s[j] = 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = fmaxf(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
#pragma unroll
          for (int j = 8; j < kN; j += 2)
            mx[j / 2 & 3] = max3(mx[j / 2 & 3], __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
          const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
          float f = 1.0f;
          const bool grow = ref == -INFINITY ? top > -INFINITY : (top - ref) * c2 > kGrow;
          if (grow) {
            f = ref == -INFINITY ? 0.0f : ex2((ref - top) * c2);
            ref = top;
            sum *= f;
          }
          if (acc && __any_sync(kAll, grow && valid)) {
            // The accumulator's last product has to be done.  Two groups: it was issued before this tile's scores,
            // so it is.  One group: it may still run.
            if (kGroups == 1) {
              warp_wait(wait, o_full(buf ^ 1), o_phase >> (buf ^ 1) & 1 ^ 1);
              fence_after();
            }
#pragma unroll 1
            for (int x = 0; x < D / 32; ++x) {
              uint32_t o[32];
              tmem_ld32(o_addr + 32 * x, o);
              wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st32(o_addr + 32 * x, o);
            }
          }
          const float shift = ref == -INFINITY ? 0.0f : kLift - ref * c2;
          const uint64_t cc = f2(c2, c2), sh = f2(shift, shift);
          uint64_t acc2[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < kN; j += 2) {
            const uint64_t t = f2_fma((uint64_t)s[j] | (uint64_t)s[j + 1] << 32, cc, sh);
            const float p0 = ex2(f2_lo(t)), p1 = ex2(f2_hi(t));
            acc2[(j >> 1) & 1] = f2_add(acc2[(j >> 1) & 1], f2(p0, p1));
            s[j >> 1] = pack16<BF16>(p0, p1);
          }
          const uint64_t both = f2_add(acc2[0], acc2[1]);
          sum += f2_lo(both) + f2_hi(both);
#pragma unroll
          for (int x = 0; x < kN / 64; ++x) tmem_st32(s_addr + 32 * x, s + 32 * x);
          wait_st();
        }
        if constexpr (kCareful) {
          const int tile = two ? u >> 1 : u, k0 = (w.it.t0 + sg.first + tile) * kN;
          const Shared all = shared_keys(a, G, w.it);
          const int s0 = max(w.it.lo - k0, 0), s1 = min(w.it.hi - k0, kN);
          const int e = min(max(all.lo - k0, s0), s1), b = max(min(all.hi - k0, s1), e);
          if (e > s0 || b < s1) {
            const int op = ring + (two ? 2 * tile + 1 : min(2 * tile + 2, 2 * m - 1));  // its place in the ring's order
            warp_wait(wait, full(op % kStages), op / kStages & 1);
            clean_values<D, BF16>(base + C::kSmemRing + op % kStages * C::kSlot, s0, e, b, s1, r);
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(p_full(buf));
        acc = true;
        if (kGroups == 1) o_phase ^= 1u << buf;
      }

      // ---- the segment's result
      const bool whole = sg.first == 0 && sg.last == w.it.payload();
      const bool join = kGroups == 2 && !two && U > 1;  // two groups hold sums of the same rows
      if (acc) {
        const int lb = kGroups == 2 ? grp : (U - 1) & 1;
        if (kGroups == 2) o_phase ^= 1u << lb;  // two groups: told once per segment
        warp_wait(wait, o_full(lb), o_phase >> lb & 1 ^ 1);
        fence_after();
      }
      float m2 = ref == -INFINITY ? -INFINITY : ref * c2 - kLift;  // log2 units from here on
      // partial sums: slot 0 if the CTA's first unit is in this item, else 1
      const int g_item = g_seg - w.off;
      const int slot = g_seg == st.first ? 0 : 1;
      float* part = part0 + ((size_t)blockIdx.x * 2 + slot) * kPartFloats;
      bool writes = two || grp == 0;  // this group puts out columns
      int col0 = 0, col1 = D;
      float f_own = 1.0f, f_other = 0.0f;
      if (join) {  // both groups' accumulators are in reach of either: each puts out half of the columns
        xch[grp * 128 + r] = make_float2(m2, sum);
        fence_before();
        named_sync(1, 256);
        fence_after();
        const float2 other = xch[(grp ^ 1) * 128 + r];
        const float M = fmaxf(m2, other.x);
        f_own = m2 == -INFINITY ? 0.0f : ex2(m2 - M);
        f_other = other.x == -INFINITY ? 0.0f : ex2(other.x - M);
        // the same sum in both groups, to the bit
        const float a0 = grp ? other.y : sum, b0 = grp ? f_other : f_own, a1 = grp ? sum : other.y, b1 = grp ? f_own : f_other;
        sum = a0 * b0 + a1 * b1;
        m2 = M;
        writes = true;
        col0 = grp * (D / 2);
        col1 = col0 + D / 2;
      }
      const float inv = inverse_of(sum);
      // the item's parts are the consecutive CTAs c0 .. c1; they join it when their own work is done
      const int c0 = whole ? 0 : st.parts ? st.c0 : owner(st, g_item + kItemUnits);
      const int parts = whole ? 1 : st.parts ? st.parts : owner(st, g_item + w.it.cost() - 1) - c0 + 1;
      const bool by_row = part_by_row(w.it.rows, parts);
      const int part_cs = by_row ? 1 : w.it.rows, part_rs = by_row ? D / 4 : 1;
      const uint32_t other_addr = lanes + C::kColO + (grp ^ 1) * D;
      const bool mixed = !kCareful && w.it.s.n > 1;  // keys that not every row sees
      uint64_t zero = 0;                             // 0 while every output is finite
      if (writes) {
        constexpr int kW = kGroups == 1 ? 64 : 32;  // columns at a time
#pragma unroll 1
        for (int x0 = col0; x0 < col1; x0 += kW) {
          uint32_t o[kW];
          if (busy && acc) {
#pragma unroll
            for (int y = 0; y < kW; y += 32) tmem_ld32(o_addr + x0 + y, o + y);
            if (join) {
              uint32_t e[kW];
#pragma unroll
              for (int y = 0; y < kW; y += 32) tmem_ld32(other_addr + x0 + y, e + y);
              wait_ld();
#pragma unroll
              for (int j = 0; j < kW; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * f_own + __uint_as_float(e[j]) * f_other);
            } else {
              wait_ld();
            }
          } else {
#pragma unroll
            for (int j = 0; j < kW; ++j) o[j] = 0u;
          }
          if (mixed) {
#pragma unroll
            for (int j = 0; j < kW; j += 2) zero = f2_fma((uint64_t)o[j] | (uint64_t)o[j + 1] << 32, 0, zero);
          }
          if (valid) {
            if (whole) {
              uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)(w.it.s.q0 + tok) * a.o_stride +
                              (int64_t)(w.it.h * G + g) * a.o_head_stride + x0;
#pragma unroll
              for (int j = 0; j < kW / 2; ++j)
                o[j] = pack16<BF16>(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
              if (wide_out) {
#pragma unroll
                for (int j = 0; j < kW / 2; j += 8) store32(out + 2 * j, o + j);
              } else {
#pragma unroll
                for (int j = 0; j < kW / 2; j += 4)
                  *reinterpret_cast<uint4*>(out + 2 * j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
              }
            } else {
              float4* dst = reinterpret_cast<float4*>(part + 2 * kRows) + x0 / 4 * part_cs + row * part_rs;
#pragma unroll
              for (int j = 0; j < kW; j += 4)
                dst[j / 4 * part_cs] = make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]),
                                                 __uint_as_float(o[j + 2]), __uint_as_float(o[j + 3]));
            }
          }
          __syncwarp();
        }
        if constexpr (kCareful) {
          const int key0 = (w.it.t0 + sg.first) * kN;
          if (valid)
            add_cleared<BF16>(a, w.it.b, w.it.h, max(lo, key0), min(hi, key0 + m * kN), shared_keys(a, G, w.it), col0, col1,
                              whole ? static_cast<uint16_t*>(a.out) + (int64_t)(w.it.s.q0 + tok) * a.o_stride +
                                          (int64_t)(w.it.h * G + g) * a.o_head_stride
                                    : nullptr,
                              part + 2 * kRows + (size_t)row * part_rs * 4, part_cs);
        } else if (mixed && valid && f2_lo(zero) + f2_hi(zero) != 0.0f && sum - sum == 0.0f) {
          st.again = 1;  // not finite, though the weights are
        }
      }
      ring += 2 * m;
      fence_before();
      writes = two || grp == 0;  // the row's statistics are written once
      if (writes && whole && valid && a.lse)
        a.lse[(int64_t)(w.it.s.q0 + tok) * a.Hq + w.it.h * G + g] =
            lse_of(m2, sum);
      if (!whole) {
        if (writes && valid) {
          reinterpret_cast<float2*>(part)[row] = make_float2(m2, sum);
        }
        if (tid == 0) {
          Cut& cut = st.cut[st.n_cut++];
          cut.c0 = c0;
          cut.parts = parts;
          cut.slot0 = st.parts || share(st, c0) >= g_item ? 0 : 1;
          cut.rows = w.it.rows;
          cut.r0 = w.it.r0;
          cut.q0 = w.it.s.q0;
          cut.h = w.it.h;
        }
      }
      if (join) named_sync(1, 256);  // both groups' columns are read before the next item's products
      g_seg += sg.len;
      walk_next<kN, kRows>(a, G, w, sg.len);
    }
  };

  // The end of a pass, for every warp: whether there is another one, on barriers of its own (the last arrivals on this
  // pass's may still be under way).
  const auto another = [&](bool careful) {
    __syncwarp();
    fence_before();
    named_sync(0, C::kThreads);
    fence_after();
    if (careful || !st.again || st.abort) return false;
    named_sync(0, C::kThreads);
    bars += C::kBars;
    if (warp == kWarpMma && lane == 0) {
      init_barriers();
      st.n_cut = 0;
    }
    named_sync(0, C::kThreads);
    return true;
  };
  // ---- the warps that feed the softmax groups
  const auto feed = [&] {
    if (warp == kWarpLoad) {
      // ---- keys and values by TMA, a box per (page, 64 columns)
      // (Page and box sizes are powers of two; what a tile's keys and values share is formed once, and the next tile's
      // page is asked for before this one's slots are waited for: with divisions and the page on the spot the copies
      // were the bound where a key tile serves 128 rows or fewer, an 8192-token prompt at head size 256 1175 us, now
      // 950.  One thread for all boxes of a tile was slower: 38 decoded tokens over 8192 keys of 64 79 us against 60.)
      const int ps = a.kv.page_size, page_log = 31 - __clz(ps);
      const int box_rows = min(ps, kN), box_log = 31 - __clz(box_rows);
      const uint32_t box_bytes = (uint32_t)box_rows * 128;
      const int part = lane % C::kSub, box = lane / C::kSub;  // this lane's box of a tile
      const uint32_t my_dst = base + C::kSmemRing + part * (kN * 128) + box * box_bytes;
      uint32_t n_ops = 0, slot = 0, phase = 1;  // of the ring: the first round's slots are free
      bool ok = true;
      struct Tile {
        uint32_t bytes;  // of the boxes that hold a visible key
        int row, page;   // this lane's box: first row of its page
        bool mine;
      };
      for (Walk w = walk_begin(st); w.left > 0 && ok;) {
        const Seg sg = walk_seg(w);
        // The ring's order: items of two row tiles consume K0 V0 K1 V1 .., the others run one tile ahead, K0 K1 V0 K2 V1
        // .. V(m-1).
        const int m = sg.tiles, lag = kGroups == 2 && w.it.rows > 128 ? 0 : 1;
        const int32_t* table = a.table + (int64_t)w.it.b * a.kv.table_stride;
        const auto prepare = [&](int i) {
          const int k0 = (w.it.t0 + sg.first + i) * kN, first = k0 + (box << box_log);
          const int b0 = (max(w.it.lo, k0) - k0) >> box_log;
          const int b1 = (min(w.it.hi, k0 + kN) - k0 + box_rows - 1) >> box_log;
          Tile x;
          x.bytes = box_bytes * (uint32_t)((b1 - b0) * C::kSub);
          x.row = first & (ps - 1);
          x.mine = box >= b0 && box < b1;
          x.page = x.mine ? __ldg(table + (first >> page_log)) : 0;
          return x;
        };
        const auto copy = [&](const Tile& x, const CUtensorMap* map) {
          ok = __all_sync(kAll, wait(empty(slot), phase));
          if (!ok) return;
          if (lane == 0) bar_expect(full(slot), x.bytes);
          __syncwarp();
          if (x.mine) {
            int page = x.page;
            if (page < 0 || page >= a.kv.num_pages) {
              set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
              page = a.kv.num_pages;  // out of range: reads as zeros
            }
            tma_4d(my_dst + slot * C::kSlot, map, part * 64, x.row, w.it.h, page, full(slot));
          }
          ++n_ops;
          if (++slot == kStages) slot = 0, phase ^= 1;
        };
        Tile next{}, now{}, before{};
        if (m) next = prepare(0);
        for (int i = 0; i < m + lag && m; ++i) {
          before = now;
          now = next;
          if (i + 1 < m) next = prepare(i + 1);
          if (i < m) copy(now, &kmap);
          if (ok && i >= lag) copy(lag ? before : now, &vmap);
          if (!ok) break;
        }
        walk_next<kN, kRows>(a, G, w, sg.len);
      }
      if (!ok && lane == 0) {  // given up: the copies in flight still land before the CTA ends
        for (uint32_t o = n_ops > (uint32_t)kStages ? n_ops - kStages : 0; o < n_ops; ++o) {
          const long long t0 = clock64();
          while (!bar_try(full(o % kStages), (o / kStages) & 1) && clock64() - t0 < kWaitCycles / 8) {
          }
        }
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      // ---- the products: one thread issues them.  (With the whole warp in the
      // loop, its votes and reconvergence cost as much as the issue itself.)
      if (elect_one()) {
        const uint32_t id_s = idesc(BF16, kN, false, a.scale < 0.0f), id_o = idesc(BF16, D, true, false);
        const uint32_t q_desc = desc_k(base + C::kSmemQ), k_desc = desc_k(base + C::kSmemRing);
        const uint32_t v_desc = desc_mn(base + C::kSmemRing, kN * 128);
        uint32_t slot = 0, phase = 0;  // of the ring
        uint32_t p_phase = 0, q_phase = 0;  // bit b: parity of buffer / row tile b
        int q_tile = 0;
        uint32_t k_slot = 0, v_slot = 0;
        const auto take = [&](uint32_t& got) {  // the ring's next tile
          wait(full(slot), phase);
          got = slot;
          if (++slot == kStages) slot = 0, phase ^= 1;
        };
        for (Walk w = walk_begin(st); w.left > 0;) {
          const Seg sg = walk_seg(w);
          const int m = sg.tiles;
          const bool two = kGroups == 2 && w.it.rows > 128;
          const int U = two ? 2 * m : m;
          const auto scores = [&](int u) {  // S(u) = Q K^T
            const int odd = u & 1, qt = two ? odd : q_tile;
            if (u == 0 || (two && u == 1)) {
              wait(q_full(qt), q_phase >> qt & 1);
              q_phase ^= 1u << qt;
            }
            if (!two || !odd) take(k_slot);
            fence_after();
            const uint32_t q = q_desc + qt * (C::kQ / 16), k = k_desc + k_slot * (C::kSlot / 16);
            const uint32_t d = tmem + C::kColS + odd * kN;
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
              mma_ss(d, q + ((x / 4) * 16384 + (x % 4) * 32) / 16, k + ((x / 4) * (kN * 128) + (x % 4) * 32) / 16, kDescHi,
                     id_s, x > 0);
            mma_commit(s_full(odd));
            if (!two || odd) mma_commit(empty(k_slot));
            if (u >= U - (two ? 2 : 1)) mma_commit(q_empty(qt));
          };
          if (U > 0) scores(0);
          if (U > 1) scores(1);
          for (int u = 0; u < U; ++u) {
            const int buf = u & 1, acc_group = kGroups == 2 ? buf : 0;
            int x0 = 0, x1 = kN / 16;  // K steps that hold a visible key
            const int tile = two ? u >> 1 : u;
            if (!two || !buf) {
              take(v_slot);
              if (tile == 0 || tile == m - 1) {
                // Values next to the item's keys, in the first and the last K step: whatever they are, even NaN, they must
                // not reach a sum.
                const int k0 = (w.it.t0 + sg.first + tile) * kN, from = max(w.it.lo - k0, 0), to = min(w.it.hi - k0, kN);
                const int begin = from & ~15, end = (to + 15) & ~15;
                for (int row = begin; row < end; ++row) {
                  if (row == from) row = to;
                  if (row == end) break;
                  uint8_t* line = smem + C::kSmemRing + v_slot * C::kSlot + row * 128;
#pragma unroll
                  for (int i = 0; i < C::kSub * 8; ++i)
                    *reinterpret_cast<uint4*>(line + (i / 8) * (kN * 128) + (i % 8) * 16) = make_uint4(0, 0, 0, 0);
                }
                if (begin < from || to < end) fence_proxy();
              }
            }
            if (tile == 0 || tile == m - 1) {
              const int k0 = (w.it.t0 + sg.first + tile) * kN;
              x0 = (max(w.it.lo, k0) - k0) / 16;
              x1 = (min(w.it.hi, k0 + kN) - k0 + 15) / 16;
            }
            wait(p_full(buf), p_phase >> buf & 1);
            p_phase ^= 1u << buf;
            fence_after();
            const uint32_t v = v_desc + v_slot * (C::kSlot / 16);
            const uint32_t d = tmem + C::kColO + acc_group * D, p = tmem + C::kColS + buf * kN;
            const bool first = u < kGroups;  // the first product of this accumulator
            if (x0 == 0 && x1 == kN / 16) {
#pragma unroll
              for (int x = 0; x < kN / 16; ++x) mma_ts(d, p + x * 8, v + x * 128, kDescHi, id_o, !first || x > 0);
            } else {
              for (int x = x0; x < x1; ++x) mma_ts(d, p + x * 8, v + x * 128, kDescHi, id_o, !first || x > x0);
            }
            if (kGroups == 1 || u >= U - 2) mma_commit(o_full(buf));
            if (!two || buf) mma_commit(empty(v_slot));
            if (u + 2 < U) scores(u + 2);
          }
          if (kGroups == 2 && U > 0 && !two) q_tile ^= 1;
          walk_next<kN, kRows>(a, G, w, sg.len);
        }
        if (st.abort) {  // given up: the products in flight end before tensor memory is freed
          mma_commit(drain());
          const long long t0 = clock64();
          while (!bar_try(drain(), 0) && clock64() - t0 < kWaitCycles / 8) {
          }
        }
      }
      __syncwarp();
    } else {
      // ---- query rows, gathered by 16-byte copies into the swizzled tiles
      const int t = tid - kWarpQ * 32;
      uint32_t used = 0, q_phase = 0;  // bit t: row tile t was filled before; parity of its next release
      int q_tile = 0;
      // a thread keeps its 16-byte column and steps down the rows: no division per copy
      constexpr int kChunks = D / 8, kStep = 64 / kChunks;
      const int ch = t % kChunks;
      for (Walk w = walk_begin(st); w.left > 0;) {
        const Seg sg = walk_seg(w);
        if (sg.tiles) {
          const bool two = kGroups == 2 && w.it.rows > 128;
          const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)w.it.s.q0 * a.q_stride +
                              (int64_t)w.it.h * G * a.q_head_stride + ch * 8;
          for (int half = 0; half < (two ? 2 : 1); ++half) {
            const int qt = two ? half : q_tile;
            if (used >> qt & 1) {
              wait(q_empty(qt), q_phase >> qt & 1);
              q_phase ^= 1u << qt;
            }
            used |= 1u << qt;
            const int rows = min(128, w.it.rows - half * 128);
            const uint32_t dst = base + C::kSmemQ + qt * C::kQ + (ch >> 3) * 16384;
            int row = t / kChunks;
            int tok = (w.it.r0 + half * 128 + row) / G, g = w.it.r0 + half * 128 + row - tok * G;
#pragma unroll 4
            for (; row < rows; row += kStep) {
              cp_async16(dst + row * 128 + (((ch & 7) ^ (row & 7)) << 4), q + tok * a.q_stride + g * a.q_head_stride);
              for (g += kStep; g >= G; g -= G) ++tok;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
          }
          if (two) {  // both tiles' copies are under way before the first is waited for
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            fence_proxy();
            bar_arrive(q_full(0));
          }
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          fence_proxy();
          bar_arrive(q_full(two ? 1 : q_tile));
          if (kGroups == 2 && !two) q_tile ^= 1;
        }
        walk_next<kN, kRows>(a, G, w, sg.len);
      }
    }
  };

  // Two groups: 384 threads start with 168 registers each; the softmax groups
  // take 208, the other four warps keep 88 (256 * 208 + 128 * 88 = 384 * 168).
  if (warp >= kWarpLoad) {
    if constexpr (kGroups == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    for (bool careful = false;; careful = true) {
      feed();
      if (!another(careful)) break;
    }
  } else {
    if constexpr (kGroups == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    softmax(std::false_type{});
    if (another(false)) {
      softmax(std::true_type{});
      another(true);
    }
    unsigned* const counters = reinterpret_cast<unsigned*>(a.ws + 16);
    if (tid == 0)
      for (int x = 0; x < st.n_cut; ++x) count_up(counters + st.cut[x].c0, st.cut[x].parts * 2 - 1);
    for (int x = 0; x < st.n_cut; ++x)
      join_parts<D, BF16>(a, G, st, st.cut[x], reinterpret_cast<float*>(a.ws + kWsHead), counters, smem + C::kSmemRing);
  }
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ---------------------------------------------------------------- host side
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

// a cache as [page][head][row][D]: boxes of 64 columns x `rows` rows of one head of one page
bool make_cache_map(CUtensorMap* map, const moe_kv_desc& kv, const void* cache, int64_t row, int64_t head, int64_t page,
                    int rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const auto bytes = [&](int64_t stride) { return (cuuint64_t)(stride ? stride * 2 : kv.D * 2); };  // 0: one entry
  const cuuint64_t dims[4] = {(cuuint64_t)kv.D, (cuuint64_t)kv.page_size, (cuuint64_t)kv.Hkv, (cuuint64_t)kv.num_pages};
  const cuuint64_t strides[3] = {bytes(row), bytes(head), bytes(page)};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(map, kv.dtype == MOE_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(cache), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16>
cudaError_t launch_t(const AttnArgs& a, cudaStream_t s) {
  using C = Cfg<D>;
  auto kern = attn_kernel<D, BF16>;
  static PerDevice opted;
  cudaError_t err = cudaSuccess;
  opted([&](int) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    return err == cudaSuccess ? 1 : 0;
  });
  if (err != cudaSuccess) return err;
  CUtensorMap km, vm;
  const int rows = std::min(a.kv.page_size, (int)C::kN);
  if (!make_cache_map(&km, a.kv, a.k_cache, a.kv.k_row_stride, a.kv.k_head_stride, a.kv.k_page_stride, rows) ||
      !make_cache_map(&vm, a.kv, a.v_cache, a.kv.v_row_stride, a.kv.v_head_stride, a.kv.v_page_stride, rows))
    return cudaErrorInvalidValue;
  const int grid = std::min(num_sms(), kMaxCtas);
  note_launch();
  // cooperative: CTAs that share an item wait for one another's parts, so all of them have to be resident
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, km, vm);
}

}  // namespace

bool attn_tensor_core(const moe_kv_desc& kv) {
  const bool one_stride = (kv.k_row_stride || kv.page_size == 1) && (kv.v_row_stride || kv.page_size == 1) &&
                          (kv.k_head_stride || kv.Hkv == 1) && (kv.v_head_stride || kv.Hkv == 1) &&
                          (kv.k_page_stride || kv.num_pages == 1) && (kv.v_page_stride || kv.num_pages == 1);
  return (kv.D == 64 || kv.D == 128 || kv.D == 256) && kv.page_size >= 16 && !(kv.page_size & (kv.page_size - 1)) &&
         one_stride;
}

bool attn_units_fit(const moe_kv_desc& kv, int Hq, int T) {
  const int64_t kn = kv.D == 256 ? 64 : 128, rows = kv.D == 256 ? 128 : 256;
  const int64_t tiles = ((int64_t)T * (Hq / kv.Hkv) / rows + kv.n_seqs) * kv.Hkv;
  return tiles * ((int64_t)kv.max_pages * kv.page_size / kn + 2 + kItemUnits) < (int64_t)1 << 31;
}

size_t attn_workspace(int, int, int D) {
  if (D != 64 && D != 128 && D != 256) return 256;
  return kWsHead + (size_t)kMaxCtas * 2 * (D == 256 ? 128 : 256) * (D + 2) * 4;
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const bool bf16 = a.kv.dtype == MOE_DT_BF16;
  switch (a.kv.D) {
    case 64: return bf16 ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
    case 128: return bf16 ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
    default: return bf16 ? launch_t<256, true>(a, s) : launch_t<256, false>(a, s);
  }
}

}  // namespace moe
