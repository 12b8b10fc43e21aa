// A dense product with its epilogue: out = act(x W^T + bias) + residual, for
// any number of rows of x.
//
// What bounds it: for few rows the weights, each read once; for many the
// tensor pipe.  W's rows are the M side (128 features to a tile) and x's the N
// side (BT tokens), so a single token costs a tile of 16 columns, and W streams
// through the same kernel at every size.
//
// Inside a CTA (warp roles): one warp feeds a ring of (W, x) tiles of 64 terms
// by TMA, one thread issues the products (tcgen05, fp32 accumulators in tensor
// memory), eight warps run the epilogue, a feature of half the tokens to a
// thread: its bias is one register, and a warp's stores and residual loads of a
// token are 32 features in a row.  Residuals are asked for a chunk of tokens
// ahead, the first before the products are done.  Two accumulators, so the
// epilogue of a tile runs beside the next tile's products.
//
// Few tiles: a cluster of CTAs takes one tile, each a share of its terms, and
// the accumulators are joined through distributed shared memory: each CTA sums
// a slice of the features, in the order of the ranks, and runs their epilogue.
//
// What it measured (bf16 but for the third): one token of 5120 x 2048 7.2 us, 37 of
// 6144 x 4096 onto an fp32 residual 14 us: 3 us to the first data, 7 for the
// weights, 3 for the join and the way out; 1021 of 7001 x 2048 with gelu (fp16)
// 27 us, three rounds of tiles; 8192 of 5120 x 4096 with silu and a residual 193 to
// 198 us, 1735 to 1784 TFLOP/s, the tensor pipe 91% active.  One token of 32768 x
// 4096: 42 us, 6.4 TB/s.  Beside a library product that adds no bias, all in bf16:
// 1 x 5120 x 2048 7.2 (library 5.6), 16 x 5120 x 2048 7.6 (5.7), 37 x 6144 x 4096
// 13.5 (11.7), 256 x 5120 x 2048 10.4 (6.8), 8192 x 5120 x 4096 180 (183), and rows
// of an odd width, 1021 x 7001 x 2048, 23 (232).
//
// Every wait is bounded: after about a second a role records
// MOE_ERR_DEVICE_TIMEOUT (where a status word is given), and all roles run to
// the end without waiting; the CTA's tiles from then on are NaN.
#include <algorithm>
#include <cmath>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_overlap.cuh"
#include "moe_per_device.h"

namespace moe {
namespace {

constexpr long long kWaitCycles = 2000000000ll;  // ~1 s at 2 GHz
constexpr int kThreads = 384;                    // warps: 0 copies, 1 products, 4 .. 11 epilogue
constexpr int kM = 128, kK = 64;                 // features of a tile, terms of a stage
constexpr int kW = kM * kK * 2;                  // bytes of a W tile

template <int BT_, bool SPLIT_>
struct Cfg {
  static constexpr int BT = BT_;
  static constexpr bool kSplit = SPLIT_;
  static constexpr int kX = BT * kK * 2, kStage = kW + kX;
  static constexpr int kPitch = BT + 4;                         // floats of a feature in the join: 16-byte reads without conflicts
  static constexpr int kJoin = SPLIT_ ? (kM + 7) * kPitch * 4 : 0;  // every rank's part of a slice of up to 135 / ranks features
  static constexpr int kPerSm = BT <= 32 ? 2 : 1;               // CTAs
  static constexpr int kBudget = (kPerSm == 2 ? 112 : 225) * 1024 - 2048 - kJoin;
  static constexpr int kStages = std::min(12, kBudget / kStage);
  static constexpr int kBufs = SPLIT_ ? 1 : 2;                  // accumulators
  static constexpr int kChunk = BT == 16 ? 8 : 16;              // tokens that a thread works on at a time
  static constexpr int kCols = std::max(32, kBufs * BT);
  static constexpr int kSmemJoin = kStages * kStage, kSmemBars = kSmemJoin + kJoin;
  static constexpr int kSmem = 1024 + kSmemBars + 512;
  static_assert(kStages >= 3 && kCols <= 512 && 8 * (2 * kStages + 4) <= 512, "sizes");
};

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
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((int)acc));
}
// The same for a pair of CTAs: a copy that is counted by a barrier of either, products over both CTAs' tiles, a commit to
// the same barrier of both, an arrival at a barrier of the other.
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void mma_ss_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((int)acc));
}
__device__ __forceinline__ void bar_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// N columns of the warp's 32 lanes, one lane (feature) per thread
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float* v) {
  uint32_t r[N];
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(addr)
        : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t remote(uint32_t local, uint32_t rank) {  // the same place in another CTA
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_remote4(uint32_t to, const float* v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
               : "memory");
}
// a / b for numbers that are not negative, quick where a < 2^20: the quotient of a + 1/2 lies at least 1 / (2 b) from a
// whole number, more than its error
__device__ __forceinline__ int quotient(int a, int b) { return a < 1 << 20 ? (int)__fdividef((float)a + 0.5f, (float)b) : a / b; }
// K-major tiles of 128-byte lines, 128-byte swizzle: 8-row groups 1024 bytes apart, a step of 16 terms is 32 bytes
constexpr uint32_t kDescHi = (uint32_t)(1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr & 0x3FFFF) >> 4) | 1u << 16; }
// kind::f16, fp32 accumulation
__device__ __forceinline__ uint32_t idesc(bool bf16, int M, int N) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

struct Wait {
  volatile int* abort;
  int* status;
  uint32_t other;  // the other CTA's abort word, of a pair (else 0)
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(bar, parity)) {
      if (*abort) return false;
      if (clock64() - t0 > kWaitCycles) {
        *abort = 1;
        if (other) asm volatile("st.shared::cluster.u32 [%0], 1;\n fence.acq_rel.cluster;" ::"r"(other) : "memory");
        set_status(status, MOE_ERR_DEVICE_TIMEOUT);
        return false;
      }
    }
    return true;
  }
};

// ---------------------------------------------------------------- epilogue
template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == MOE_ACT_RELU) return v < 0.0f ? 0.0f : v;  // (NaN stays)
  else if constexpr (ACT == MOE_ACT_SILU) {  // 2^x within 2 ulp of its rounded argument, a quotient within 2 ulp
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.44269504088896341f));
    return __fdividef(v, 1.0f + e);
  }
  else if constexpr (ACT == MOE_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.707106781186547524f));
  else if constexpr (ACT == MOE_ACT_GELU_TANH)
    return 0.5f * v * (1.0f + tanhf(0.797884560802865356f * fmaf(0.044715f * v * v, v, v)));
  else return v;
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
template <typename O, int N>
__device__ __forceinline__ void store(const LinearArgs& a, int feature, int t, int n, const float* v) {
  O* p = static_cast<O*>(a.out) + t * a.o_stride + feature;
  if (n >= N) {  // (a test at each store, though never false, made an epilogue of stores alone 2.5 times as long)
#pragma unroll
    for (int i = 0; i < N; ++i) put(p + i * a.o_stride, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) put(p + i * a.o_stride, v[i]);
  }
}
template <int ACT, int N>
__device__ __forceinline__ void activate_all(float bias, float* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = activate<ACT>(v[i] + bias);
}
template <typename T, int N>
__device__ __forceinline__ void ask_rows(const T* p, int64_t stride, int n, uint32_t* raw) {
  if (n >= N) {
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = p[i * stride];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) raw[i] = p[i * stride];
  }
}
// The residual's n <= N tokens from t on of one feature, as they are stored.
template <int N>
__device__ __forceinline__ void ask_residual(const LinearArgs& a, int feature, int t, int n, uint32_t* raw) {
  if (!a.residual || feature >= a.N) return;
  const int64_t at = t * a.r_stride + feature;
  if (a.r_dtype == MOE_DT_F32) ask_rows<uint32_t, N>(static_cast<const uint32_t*>(a.residual) + at, a.r_stride, n, raw);
  else ask_rows<uint16_t, N>(static_cast<const uint16_t*>(a.residual) + at, a.r_stride, n, raw);
}
// n <= N tokens from t on of one feature: `v` their products, `raw` their residuals
template <int N>
__device__ __forceinline__ void finish(const LinearArgs& a, float bias, int feature, int t, int n, float* v, const uint32_t* raw) {
  if (feature >= a.N) return;
  switch (a.act) {
    case MOE_ACT_RELU: activate_all<MOE_ACT_RELU, N>(bias, v); break;
    case MOE_ACT_SILU: activate_all<MOE_ACT_SILU, N>(bias, v); break;
    case MOE_ACT_GELU: activate_all<MOE_ACT_GELU, N>(bias, v); break;
    case MOE_ACT_GELU_TANH: activate_all<MOE_ACT_GELU_TANH, N>(bias, v); break;
    default: activate_all<MOE_ACT_NONE, N>(bias, v);
  }
  if (a.residual) {
    if (a.r_dtype == MOE_DT_F32) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __uint_as_float(raw[i]);
    } else if (a.r_dtype == MOE_DT_BF16) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __uint_as_float(raw[i] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __half2float(__ushort_as_half((unsigned short)raw[i]));
    }
  }
  if (a.o_dtype == MOE_DT_F32) store<float, N>(a, feature, t, n, v);
  else if (a.o_dtype == MOE_DT_BF16) store<__nv_bfloat16, N>(a, feature, t, n, v);
  else store<__half, N>(a, feature, t, n, v);
}

__device__ __forceinline__ float bias_of(const LinearArgs& a, int feature) {
  return a.bias && feature < a.N ? __ldg(a.bias + feature) : 0.0f;
}
// Brings a tile's residuals to L2, 128 bytes to each of the 256 epilogue threads (`thread`) at a time.  Asked for a tile ahead:
// the way from memory takes as long as the epilogue of half a tile.
__device__ __forceinline__ void prefetch_residual(const LinearArgs& a, int feature, int t, int live, int thread) {
  if (!a.residual) return;
  const int size = a.r_dtype == MOE_DT_F32 ? 4 : 2, lines = kM * size / 128;
  for (int i = thread; i < live * lines; i += 256) {
    const int token = i / lines, f = feature + (i - token * lines) * (128 / size);
    if (f < a.N)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.residual) + ((t + token) * a.r_stride + f) * size));
  }
}
// A thread's part of a tile that is not shared: feature, tokens t .. t + live, of its accumulator's columns the half `part`;
// `ready` waits for the products and tells whether they are all there: what is written without them is NaN.
template <int BT, int CH, typename F>
__device__ __forceinline__ void finish_tile(const LinearArgs& a, uint32_t acc, int feature, int t, int live, int part, F ready) {
  uint32_t raw[2][CH];
  const int c0 = part * (BT / 2), c1 = min(live, c0 + BT / 2);
  float bias = bias_of(a, feature);
  if (c0 < c1) ask_residual<CH>(a, feature, t + c0, c1 - c0, raw[0]);
  if (!ready()) bias = NAN;
#pragma unroll 1
  for (int c = c0; c < c1; c += CH) {
    if (c + CH < c1) ask_residual<CH>(a, feature, t + c + CH, c1 - c - CH, raw[1]);
    float v[CH];
    __syncwarp();
    tmem_ld<CH>(acc + c, v);
    finish<CH>(a, bias, feature, t + c, c1 - c, v, raw[0]);
#pragma unroll
    for (int x = 0; x < CH; ++x) raw[0][x] = raw[1][x];
  }
}

// A tile's place among f_tiles x t_tiles: the tokens of a group of kGroup feature tiles before the next group, so that what
// runs at one time shares both sides' tiles in L2.
template <int kGroup>
__device__ __forceinline__ void tile_of(int i, int f_tiles, int t_tiles, int& f, int& t) {
  const int g = quotient(i, kGroup * t_tiles), in = i - g * kGroup * t_tiles, n = min(kGroup, f_tiles - g * kGroup);
  t = quotient(in, n);
  f = g * kGroup + in - t * n;
}

template <class C>
__global__ void __launch_bounds__(kThreads, C::kPerSm) linear_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap wm,
                                                                     const __grid_constant__ CUtensorMap xm) {
  constexpr int BT = C::BT, kStages = C::kStages, kBufs = C::kBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023);  // the swizzled tiles start on 1024-byte boundaries
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t base = smem_u32(smem), bars = base + C::kSmemBars;
  const auto full = [&](int s) { return bars + s * 8; };
  const auto empty = [&](int s) { return bars + (kStages + s) * 8; };
  const auto acc_full = [&](int b) { return bars + (2 * kStages + b) * 8; };
  const auto acc_empty = [&](int b) { return bars + (2 * kStages + 2 + b) * 8; };
  const int ranks = C::kSplit ? a.split : 1, rank = C::kSplit ? (int)cluster_rank() : 0;
  const int blocks = (a.K + kK - 1) / kK;
  const int k0 = quotient(rank * blocks, ranks), k1 = quotient((rank + 1) * blocks, ranks);
  const int f_tiles = (a.N + kM - 1) / kM, t_tiles = (a.T + BT - 1) / BT;
  const int tiles = f_tiles * t_tiles, first = quotient(blockIdx.x, ranks);
  const int step = C::kSplit ? tiles : gridDim.x;

  const auto tile_at = [&](int i, int& f, int& t) { tile_of<16>(i, f_tiles, t_tiles, f, t); };
  const auto copy = [&](int s, int k, int f, int t) {
    bar_expect(full(s), C::kStage);
    tma_2d(base + s * C::kStage, &wm, k * kK, f * kM, full(s));
    tma_2d(base + s * C::kStage + kW, &xm, k * kK, t * BT, full(s));
  };

  const int ahead = min(kStages, k1 - k0);  // stages of the first tile that are asked for before anything else
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) bar_init(full(s), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    int f, t;
    tile_at(first, f, t);
    wait_for_previous();
    for (int s = 0; s < ahead; ++s) copy(s, k0 + s, f, t);
  }
  if (tid == 32) {
    for (int s = 0; s < kStages; ++s) bar_init(empty(s), 1);
    for (int b = 0; b < 2; ++b) bar_init(acc_full(b), 1), bar_init(acc_empty(b), 8);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "n"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  wait_for_previous();
  fence_before();
  __syncthreads();
  fence_after();
  let_next_start();  // (this CTA has its tensor memory: one of the next kernel can no longer take it and wait for this one)
  if (C::kSplit) cluster_arrive();  // this CTA runs: others may write to it once they have waited
  const uint32_t tmem = s_tmem;
  const Wait wait{&s_abort, a.status, 0};
  if (warp == 0) {
    if (elect_one()) {
      int s = ahead == kStages ? 0 : ahead;
      uint32_t parity = ahead == kStages ? 0 : 1;  // of the ring's empty barriers: the first round does not wait
      for (int i = first; i < tiles; i += step) {
        int f, t;
        tile_at(i, f, t);
        for (int k = i == first ? k0 + ahead : k0; k < k1; ++k) {
          if (!wait(empty(s), parity)) break;
          copy(s, k, f, t);
          if (++s == kStages) s = 0, parity ^= 1;
        }
        if (s_abort) break;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      int s = 0, buf = 0;
      uint32_t parity = 0, acc_parity = 1;
      const uint32_t id = idesc(a.x_dtype == MOE_DT_BF16, kM, BT);
      for (int i = first; i < tiles; i += step) {
        if (!wait(acc_empty(buf), acc_parity)) break;
        fence_after();
        for (int k = k0; k < k1; ++k) {
          if (!wait(full(s), parity)) break;
          fence_after();
          const uint32_t w = desc_k(base + s * C::kStage), x = desc_k(base + s * C::kStage + kW);
#pragma unroll
          for (int j = 0; j < kK / 16; ++j) mma_ss(tmem + buf * BT, w + 2 * j, x + 2 * j, kDescHi, id, k > k0 || j > 0);
          mma_commit(empty(s));
          if (++s == kStages) s = 0, parity ^= 1;
        }
        mma_commit(acc_full(buf));
        if (++buf == kBufs) buf = 0, acc_parity ^= 1;
        if (s_abort) break;
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    int buf = 0;
    uint32_t acc_parity = 0;
    constexpr int CH = C::kChunk;
    const int row = tid & 127, part = (tid >> 7) - 1;  // of the tile: a feature, and one of two parts of the tokens
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    for (int i = first; i < tiles; i += step) {
      int f, t;
      tile_at(i, f, t);
      const int feature = f * kM + row, live = min(BT, a.T - t * BT);  // tokens of the tile
      const uint32_t acc = tmem + lanes + buf * BT;
      if constexpr (C::kSplit) {
        // slice r of the features goes to rank r: [from rank][feature of the slice][token]
        const int lo = rank * kM / ranks, nf = (rank + 1) * kM / ranks - lo;       // this rank's
        const int to = ((row + 1) * ranks - 1) / kM, to_lo = to * kM / ranks, to_nf = (to + 1) * kM / ranks - to_lo;
        const uint32_t dst = remote(base + C::kSmemJoin + (rank * to_nf + row - to_lo) * (C::kPitch * 4), to);
        // Of the join a thread takes 4 tokens of one feature at a time, lanes next to each other features.  This code runs
        // once, so it is kept short rather than unrolled (16 tokens at a time: 1 us more, for instructions that are fetched
        // for the first time), and the residuals are brought to the first cache meanwhile instead of to registers.
        const int groups = quotient(256, nf), q0 = quotient(tid - 128, nf), fi = tid - 128 - q0 * nf;
        const int quads = q0 < groups ? (live + 3) / 4 : 0, mine = f * kM + lo + fi;
        const float bias = bias_of(a, mine);
        if (a.residual && mine < a.N) {
          const int size = a.r_dtype == MOE_DT_F32 ? 4 : 2;
          const char* p = static_cast<const char*>(a.residual) + ((int64_t)t * BT * a.r_stride + mine) * size;
#pragma unroll 1
          for (int q = q0; q < quads; q += groups)
            for (int x = 4 * q; x < min(4 * q + 4, live); ++x)
              asm volatile("prefetch.global.L1 [%0];" ::"l"(p + x * a.r_stride * size));
        }
        wait(acc_full(buf), acc_parity);
        __syncwarp();
        fence_after();
        cluster_wait();
        for (int c = part * CH; c < live; c += 2 * CH) {
          float v[CH];
          __syncwarp();
          tmem_ld<CH>(acc + c, v);
          if (s_abort) {
#pragma unroll
            for (int x = 0; x < CH; ++x) v[x] = NAN;
          }
#pragma unroll
          for (int x = 0; x < CH; x += 4)
            if (c + x < live) store_remote4(dst + (c + x) * 4, v + x);
        }
        cluster_arrive();
        cluster_wait();
        const float* const join = reinterpret_cast<const float*>(smem + C::kSmemJoin);
#pragma unroll 1
        for (int q = q0; q < quads; q += groups) {
          uint32_t raw[4];
          ask_residual<4>(a, mine, t * BT + 4 * q, live - 4 * q, raw);
          float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int r = 0; r < ranks; ++r) {
            const float4 w = *reinterpret_cast<const float4*>(join + (r * nf + fi) * C::kPitch + 4 * q);
            v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
          }
          finish<4>(a, bias, mine, t * BT + 4 * q, live - 4 * q, v, raw);
        }
      } else {
        if (i == first) prefetch_residual(a, f * kM, t * BT, live, tid - 128);
        if (i + step < tiles) {
          int nf, nt;
          tile_at(i + step, nf, nt);
          prefetch_residual(a, nf * kM, nt * BT, min(BT, a.T - nt * BT), tid - 128);
        }
        finish_tile<BT, CH>(a, acc, feature, t * BT, live, part, [&] {
          wait(acc_full(buf), acc_parity);
          __syncwarp();
          fence_after();
          return !s_abort;
        });
      }
      fence_before();
      __syncwarp();
      if ((tid & 31) == 0) bar_arrive(acc_empty(buf));
      if (++buf == kBufs) buf = 0, acc_parity ^= 1;
    }
  }
  if (C::kSplit && warp < 4) {  // the epilogue warps' three meetings
    cluster_wait();
    cluster_arrive();
    cluster_wait();
  }
  if (s_abort) {  // copies and products may be in flight still
    const long long t0 = clock64();
    while (clock64() - t0 < kWaitCycles / 8) {
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kCols));
  }
}

// ---------------------------------------------------------------- pairs of CTAs
// Many tokens: two CTAs on neighbouring SMs form products over 256 features and BT tokens.  Each holds the W tile of its 128
// features and the x tile of half the tokens, and the tensor pipes of both read both halves, so an SM takes 64 bytes per
// clock at BT = 256.  Alone it takes 96 for its products, and gets 75: 8192 tokens of 5120 x 4096 were bound by that.
template <int BT_>
struct PairCfg {
  static constexpr int BT = BT_;
  static constexpr int kX = BT / 2 * kK * 2, kStage = kW + kX;  // of each CTA
  static constexpr int kStages = std::min(9, (225 * 1024 - 2048) / kStage);
  static constexpr int kCols = 2 * BT;
  static constexpr int kSmemBars = kStages * kStage;
  static constexpr int kSmem = 1024 + kSmemBars + 512;
  static_assert(kCols <= 512 && 8 * (2 * kStages + 4) <= 512, "sizes");
};

template <class C>
__global__ void __launch_bounds__(kThreads, 1) linear_pair_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap wm,
                                                                  const __grid_constant__ CUtensorMap xm) {
  constexpr int BT = C::BT, kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023);
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t base = smem_u32(smem), bars = base + C::kSmemBars;
  const auto full = [&](int s) { return bars + s * 8; };               // of the leader (rank 0): both CTAs' copies
  const auto empty = [&](int s) { return bars + (kStages + s) * 8; };  // of each
  const auto acc_full = [&](int b) { return bars + (2 * kStages + b) * 8; };
  const auto acc_empty = [&](int b) { return bars + (2 * kStages + 2 + b) * 8; };  // of the leader: both CTAs' epilogues
  const int rank = (int)cluster_rank();
  const int blocks = (a.K + kK - 1) / kK;
  const int f_tiles = (a.N + 2 * kM - 1) / (2 * kM), t_tiles = (a.T + BT - 1) / BT, tiles = f_tiles * t_tiles;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) bar_init(full(s), 1), bar_init(empty(s), 1);
    for (int b = 0; b < 2; ++b) bar_init(acc_full(b), 1), bar_init(acc_empty(b), 16);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&wm)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&xm)) : "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "n"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  __syncwarp();
  wait_for_previous();
  fence_before();
  cluster_arrive();
  cluster_wait();  // both CTAs' barriers and tensor memory are there
  fence_after();
  let_next_start();
  const uint32_t tmem = s_tmem;
  const Wait wait{&s_abort, a.status, remote(smem_u32(const_cast<int*>(&s_abort)), rank ^ 1)};
  const auto tile_at = [&](int i, int& f, int& t) { tile_of<8>(i, f_tiles, t_tiles, f, t); };

  if (warp == 0) {
    if (elect_one()) {
      int s = 0;
      uint32_t parity = 1;  // of the ring's empty barriers: the first round does not wait
      for (int i = first; i < tiles; i += step) {
        int f, t;
        tile_at(i, f, t);
        for (int k = 0; k < blocks; ++k) {
          if (!wait(empty(s), parity)) break;
          const uint32_t bar = remote(full(s), 0), dst = base + s * C::kStage;
          if (rank == 0) bar_expect(full(s), 2 * C::kStage);
          tma_2d_pair(dst, &wm, k * kK, (2 * f + rank) * kM, bar);
          tma_2d_pair(dst + kW, &xm, k * kK, t * BT + rank * (BT / 2), bar);
          if (++s == kStages) s = 0, parity ^= 1;
        }
        if (s_abort) break;
      }
      // the last commits reach this CTA before it ends
      for (int j = 0; j < kStages && !s_abort; ++j) {
        wait(empty(s), parity);
        if (++s == kStages) s = 0, parity ^= 1;
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    if (elect_one()) {
      int s = 0, buf = 0;
      uint32_t parity = 0, acc_parity = 1;
      const uint32_t id = idesc(a.x_dtype == MOE_DT_BF16, 2 * kM, BT);
      for (int i = first; i < tiles; i += step) {
        if (!wait(acc_empty(buf), acc_parity)) break;
        fence_after();
        for (int k = 0; k < blocks; ++k) {
          if (!wait(full(s), parity)) break;
          fence_after();
          const uint32_t w = desc_k(base + s * C::kStage), x = desc_k(base + s * C::kStage + kW);
#pragma unroll
          for (int j = 0; j < kK / 16; ++j) mma_ss_pair(tmem + buf * BT, w + 2 * j, x + 2 * j, kDescHi, id, k > 0 || j > 0);
          mma_commit_pair(empty(s));
          if (++s == kStages) s = 0, parity ^= 1;
        }
        mma_commit_pair(acc_full(buf));
        buf ^= 1;
        if (!buf) acc_parity ^= 1;
        if (s_abort) break;
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    int buf = 0;
    uint32_t acc_parity = 0;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    for (int i = first; i < tiles; i += step) {
      int f, t;
      tile_at(i, f, t);
      if (i == first) prefetch_residual(a, (2 * f + rank) * kM, t * BT, min(BT, a.T - t * BT), tid - 128);
      if (i + step < tiles) {
        int nf, nt;
        tile_at(i + step, nf, nt);
        prefetch_residual(a, (2 * nf + rank) * kM, nt * BT, min(BT, a.T - nt * BT), tid - 128);
      }
      finish_tile<BT, 16>(a, tmem + lanes + buf * BT, (2 * f + rank) * kM + (tid & 127), t * BT, min(BT, a.T - t * BT),
                          (tid >> 7) - 1, [&] {
                            wait(acc_full(buf), acc_parity);
                            __syncwarp();
                            fence_after();
                            return !s_abort;
                          });
      fence_before();
      __syncwarp();
      if ((tid & 31) == 0) bar_arrive_remote(remote(acc_empty(buf), 0));
      buf ^= 1;
      if (!buf) acc_parity ^= 1;
    }
  }
  if (s_abort) {  // copies and products may be in flight still
    const long long t0 = clock64();
    while (clock64() - t0 < kWaitCycles / 8) {
    }
  }
  __syncwarp();
  fence_before();
  cluster_arrive();
  cluster_wait();  // the other CTA reads no tile of this one any more, and signals no barrier
  if (warp == 2) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kCols));
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
// rows of K elements: boxes of 64 elements x `rows` rows; what lies outside reads as zeros
bool make_map(CUtensorMap* map, int dtype, const void* p, int64_t rows, int K, int64_t stride, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(rows > 1 ? stride : K) * 2};
  const cuuint32_t box[2] = {kK, (cuuint32_t)box_rows}, one[2] = {1, 1};
  return fn(map, dtype == MOE_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sets a kernel up once per device.
template <class C>
cudaError_t opt_in() {
  static PerDevice opted;
  cudaError_t err = cudaSuccess;
  opted([&](int) {
    err = cudaFuncSetAttribute(linear_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    return err == cudaSuccess ? 1 : 0;
  });
  return err;
}
// Tiles of `split` CTAs each that the device holds at one time: clusters stay within a group of SMs, so they leave some idle.
template <int BT>
int room(int split) {
  if (split == 1) return Cfg<BT, false>::kPerSm * num_sms();
  if constexpr (BT <= 128) {
    using C = Cfg<BT, true>;
    static PerDevice kept[9];
    return kept[split]([&](int) {
      cudaLaunchAttribute attr{};
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = (unsigned)split;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3((unsigned)split);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = C::kSmem;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (opt_in<C>() != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, linear_kernel<C>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
      }
      return n;
    });
  }
  return 0;
}

template <class C>
cudaError_t launch_t(LinearArgs a, int split, cudaStream_t s) {
  const cudaError_t err = opt_in<C>();
  if (err != cudaSuccess) return err;
  CUtensorMap wm, xm;
  if (!make_map(&wm, a.x_dtype, a.w, a.N, a.K, a.w_stride, kM) || !make_map(&xm, a.x_dtype, a.x, a.T, a.K, a.x_stride, C::BT))
    return cudaErrorInvalidValue;
  a.split = split;
  const int64_t tiles = (int64_t)((a.N + kM - 1) / kM) * ((a.T + C::BT - 1) / C::BT);
  const int64_t grid = C::kSplit ? tiles * split : std::min<int64_t>(tiles, (int64_t)C::kPerSm * num_sms());
  note_launch();
  return launch_overlapping(linear_kernel<C>, dim3((unsigned)grid), kThreads, C::kSmem, split, s, a, wm, xm);
}
template <int BT>
cudaError_t launch_tokens(const LinearArgs& a, int split, cudaStream_t s) {
  if constexpr (BT <= 128) {
    if (split > 1) return launch_t<Cfg<BT, true>>(a, split, s);
  }
  return launch_t<Cfg<BT, false>>(a, 1, s);
}

template <int BT>
cudaError_t launch_pair(const LinearArgs& a, cudaStream_t s) {
  using C = PairCfg<BT>;
  static PerDevice opted;
  cudaError_t err = cudaSuccess;
  opted([&](int) {
    err = cudaFuncSetAttribute(linear_pair_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    return err == cudaSuccess ? 1 : 0;
  });
  if (err != cudaSuccess) return err;
  CUtensorMap wm, xm;
  if (!make_map(&wm, a.x_dtype, a.w, a.N, a.K, a.w_stride, kM) || !make_map(&xm, a.x_dtype, a.x, a.T, a.K, a.x_stride, BT / 2))
    return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)((a.N + 2 * kM - 1) / (2 * kM)) * ((a.T + BT - 1) / BT);
  note_launch();
  return launch_overlapping(linear_pair_kernel<C>, dim3((unsigned)(2 * std::min<int64_t>(tiles, num_sms() / 2))), kThreads, C::kSmem, 2,
                            s, a, wm, xm);
}

// The least of all tiles and divisions by what they cost (bt, split; split 0: pairs of CTAs), in clocks: rounds of the tiles,
// each a number of stages that wait for the products or for the copies into an SM, and the last epilogue.  The constants are
// fits to measured times; with tiles and divisions forced, in us (bf16, bias):
//                              64     64, 2 CTAs   128    128, 3 CTAs    256   pairs 128   pairs 256
//    37 x  6144 x 4096       14.9         14.9    19.3           24.6      -           -           -
//   100 x  5120 x 2048        9.0            -    11.6           12.4   16.4        11.1        15.3
//  1021 x  7001 x 2048       33.2            -    26.8              -   29.8        24.7        27.2
//  4096 x  2048 x 1024       23.0            -    19.7              -   19.0        20.1        17.7
//  8192 x  5120 x 4096        325            -     235              -    228         207         187
struct Choice {
  int bt, split;
  double cost;
};
double epilogue_cost(const LinearArgs& a, int bt) {  // of a tile
  const double act = a.act == MOE_ACT_SILU ? 12 : a.act == MOE_ACT_GELU ? 35 : a.act == MOE_ACT_GELU_TANH ? 27 : 0;
  return std::min(bt, a.T) * (20.0 + act + (a.residual ? 30.0 : 0.0));
}
template <int BT>
void consider_pair(const LinearArgs& a, Choice& best) {
  const int blocks = (a.K + kK - 1) / kK;
  const int64_t tiles = (int64_t)((a.N + 2 * kM - 1) / (2 * kM)) * ((a.T + BT - 1) / BT);
  const double rounds = std::ceil((double)tiles / (num_sms() / 2));
  const double stage = std::max(2.0 * BT, PairCfg<BT>::kStage / 75.0);
  const double cost = rounds * blocks * stage + epilogue_cost(a, BT) + 4500.0;
  if (cost < best.cost) best = Choice{BT, 0, cost};
}
template <int BT>
void consider(const LinearArgs& a, Choice& best) {
  const int blocks = (a.K + kK - 1) / kK, sms = num_sms();
  const int64_t tiles = (int64_t)((a.N + kM - 1) / kM) * ((a.T + BT - 1) / BT);
  for (int split = 1; split <= (BT <= 128 ? 8 : 1) && split <= std::max(1, blocks / 2); ++split) {
    const int hold = room<BT>(split);
    if (split > 1 && tiles > hold) continue;
    const double bytes = kW + BT * 128.0;
    const int64_t ctas = std::min<int64_t>(tiles, hold) * split;
    const int on_sm = (int)std::min<int64_t>(Cfg<BT, false>::kPerSm, (ctas + sms - 1) / sms);
    const double rounds = std::ceil((double)tiles / hold), per = (double)((blocks + split - 1) / split);
    const double stage = std::max({2.0 * BT * on_sm, bytes * on_sm / 60.0, bytes * ctas / 8000.0});
    const double cost = rounds * per * stage + epilogue_cost(a, BT) + (split > 1 ? 2000.0 + 60.0 * std::min(BT, a.T) : 0.0);
    if (cost < best.cost) best = Choice{BT, split, cost};
  }
}

}  // namespace

bool linear_plan_ok(LinearPlan p, int T, int N, int K) {
  const int t = p.tokens, blocks = (K + kK - 1) / kK;
  if (t != 16 && t != 32 && t != 64 && t != 128 && t != 256) return false;
  if (p.ctas < 0 || p.ctas > 8 || (p.ctas == 0 && t < 128) || (p.ctas > 1 && (t > 128 || p.ctas > blocks))) return false;
  return ((int64_t)N / kM + 1) * ((int64_t)T / t + 1) < 1 << 24;  // (a split's CTAs are the grid)
}

cudaError_t launch_linear(const LinearArgs& a, LinearPlan p, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (p.tokens == 0) {
    Choice c{256, 1, 1e300};
    consider<16>(a, c);
    consider<32>(a, c);
    consider<64>(a, c);
    consider<128>(a, c);
    consider<256>(a, c);
    consider_pair<128>(a, c);
    consider_pair<256>(a, c);
    p = LinearPlan{c.bt, c.split};
  }
  if (p.ctas == 0) return p.tokens == 128 ? launch_pair<128>(a, s) : launch_pair<256>(a, s);
  switch (p.tokens) {
    case 16: return launch_tokens<16>(a, p.ctas, s);
    case 32: return launch_tokens<32>(a, p.ctas, s);
    case 64: return launch_tokens<64>(a, p.ctas, s);
    case 128: return launch_tokens<128>(a, p.ctas, s);
    default: return launch_tokens<256>(a, 1, s);
  }
}

}  // namespace moe
