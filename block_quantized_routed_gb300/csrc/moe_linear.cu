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
// memory), four warps run the epilogue, a feature to a thread: its bias is one
// register, and a warp's stores and residual loads of a token are 32 features
// in a row.  Two accumulators, so the epilogue of a tile runs beside the next
// tile's products.
//
// Few tiles: a cluster of CTAs takes one tile, each a share of its terms, and
// the accumulators are joined through distributed shared memory: each CTA sums
// a slice of the tokens, in the order of the ranks, and runs their epilogue.
//
// Every wait is bounded: after about a second a role records
// MOE_ERR_DEVICE_TIMEOUT (where a status word is given), and all roles run to
// the end without waiting.
#include <algorithm>
#include <cmath>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_per_device.h"

namespace moe {
namespace {

constexpr long long kWaitCycles = 2000000000ll;  // ~1 s at 2 GHz
constexpr int kThreads = 256;                    // warps: 0 copies, 1 products, 4 .. 7 epilogue
constexpr int kM = 128, kK = 64;                 // features of a tile, terms of a stage
constexpr int kW = kM * kK * 2;                  // bytes of a W tile

template <int BT_, bool SPLIT_>
struct Cfg {
  static constexpr int BT = BT_;
  static constexpr bool kSplit = SPLIT_;
  static constexpr int kX = BT * kK * 2, kStage = kW + kX;
  static constexpr int kJoin = SPLIT_ ? (BT + 8) * kM * 4 : 0;  // every rank's accumulators of a slice: up to (BT + 7) / ranks tokens each
  static constexpr int kPerSm = BT <= 32 ? 2 : 1;               // CTAs
  static constexpr int kBudget = (kPerSm == 2 ? 112 : 225) * 1024 - 2048 - kJoin;
  static constexpr int kStages = std::min(12, kBudget / kStage);
  static constexpr int kBufs = SPLIT_ ? 1 : 2;                  // accumulators
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
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 16 columns of the warp's 32 lanes, one lane (feature) per thread
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void store_remote(uint32_t local, uint32_t rank, float v) {  // the same place in another CTA
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.f32 [a], %2;\n}\n" ::"r"(local),
               "r"(rank), "f"(v)
               : "memory");
}
// K-major tiles of 128-byte lines, 128-byte swizzle: 8-row groups 1024 bytes apart, a step of 16 terms is 32 bytes
constexpr uint32_t kDescHi = (uint32_t)(1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr & 0x3FFFF) >> 4) | 1u << 16; }
// kind::f16, fp32 accumulation, M = 128
__device__ __forceinline__ uint32_t idesc(bool bf16, int N) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (uint32_t)(N >> 3) << 17 | (uint32_t)(kM >> 4) << 24;
}

struct Wait {
  volatile int* abort;
  int* status;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(bar, parity)) {
      if (*abort) return false;
      if (clock64() - t0 > kWaitCycles) {
        *abort = 1;
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
  else if constexpr (ACT == MOE_ACT_SILU) return v / (1.0f + expf(-v));
  else if constexpr (ACT == MOE_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.707106781186547524f));
  else if constexpr (ACT == MOE_ACT_GELU_TANH)
    return 0.5f * v * (1.0f + tanhf(0.797884560802865356f * fmaf(0.044715f * v * v, v, v)));
  else return v;
}
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
template <typename R, int N>
__device__ __forceinline__ void add_residual(const LinearArgs& a, int feature, int t, float* v) {
  const R* p = static_cast<const R*>(a.residual) + t * a.r_stride + feature;
  R r[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (t + i < a.T) r[i] = p[i * a.r_stride];
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (t + i < a.T) v[i] += to_f(r[i]);
}
template <typename O, int N>
__device__ __forceinline__ void store(const LinearArgs& a, int feature, int t, const float* v) {
  O* p = static_cast<O*>(a.out) + t * a.o_stride + feature;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (t + i < a.T) put(p + i * a.o_stride, v[i]);
}
// N tokens from t on of one feature: `v` their products
template <int ACT, int N>
__device__ __forceinline__ void activate_all(float bias, float* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = activate<ACT>(v[i] + bias);
}
template <int N>
__device__ __forceinline__ void finish(const LinearArgs& a, float bias, int feature, int t, float* v) {
  if (feature >= a.N) return;
  switch (a.act) {
    case MOE_ACT_RELU: activate_all<MOE_ACT_RELU, N>(bias, v); break;
    case MOE_ACT_SILU: activate_all<MOE_ACT_SILU, N>(bias, v); break;
    case MOE_ACT_GELU: activate_all<MOE_ACT_GELU, N>(bias, v); break;
    case MOE_ACT_GELU_TANH: activate_all<MOE_ACT_GELU_TANH, N>(bias, v); break;
    default: activate_all<MOE_ACT_NONE, N>(bias, v);
  }
  if (a.residual) {
    if (a.r_dtype == MOE_DT_F32) add_residual<float, N>(a, feature, t, v);
    else if (a.r_dtype == MOE_DT_BF16) add_residual<__nv_bfloat16, N>(a, feature, t, v);
    else add_residual<__half, N>(a, feature, t, v);
  }
  if (a.o_dtype == MOE_DT_F32) store<float, N>(a, feature, t, v);
  else if (a.o_dtype == MOE_DT_BF16) store<__nv_bfloat16, N>(a, feature, t, v);
  else store<__half, N>(a, feature, t, v);
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
  const int k0 = rank * blocks / ranks, k1 = (rank + 1) * blocks / ranks;
  const int f_tiles = (a.N + kM - 1) / kM, t_tiles = (a.T + BT - 1) / BT;
  const int tiles = f_tiles * t_tiles, first = blockIdx.x / ranks, step = gridDim.x / ranks;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) bar_init(full(s), 1), bar_init(empty(s), 1);
    for (int b = 0; b < 2; ++b) bar_init(acc_full(b), 1), bar_init(acc_empty(b), 4);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&wm)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&xm)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "n"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (C::kSplit) cluster_arrive();  // this CTA runs: others may write to it once they have waited
  const uint32_t tmem = s_tmem;
  const Wait wait{&s_abort, a.status};
  // a tile's first feature and token: the tokens of a group of feature tiles before the next group, so that what
  // runs at one time shares both sides' tiles in L2
  const auto tile_at = [&](int i, int& f, int& t) {
    constexpr int kGroup = 16;
    const int g = i / (kGroup * t_tiles), in = i - g * kGroup * t_tiles, n = min(kGroup, f_tiles - g * kGroup);
    t = in / n;
    f = g * kGroup + in - t * n;
  };

  if (warp == 0) {
    if (elect_one()) {
      int s = 0;
      uint32_t parity = 1;  // of the ring's empty barriers: the first round does not wait
      for (int i = first; i < tiles; i += step) {
        int f, t;
        tile_at(i, f, t);
        for (int k = k0; k < k1; ++k) {
          if (!wait(empty(s), parity)) break;
          bar_expect(full(s), C::kStage);
          tma_2d(base + s * C::kStage, &wm, k * kK, f * kM, full(s));
          tma_2d(base + s * C::kStage + kW, &xm, k * kK, t * BT, full(s));
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
      const uint32_t id = idesc(a.x_dtype == MOE_DT_BF16, BT);
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
    const int row = tid - 128;  // of the tile: a feature
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    for (int i = first; i < tiles; i += step) {
      int f, t;
      tile_at(i, f, t);
      const int feature = f * kM + row;
      const float bias = a.bias && feature < a.N ? __ldg(a.bias + feature) : 0.0f;
      wait(acc_full(buf), acc_parity);
      __syncwarp();
      fence_after();
      const uint32_t acc = tmem + lanes + buf * BT;
      if constexpr (C::kSplit) {
        // slice r of the tokens goes to rank r: [from rank][token of the slice][feature]
        cluster_wait();
        for (int c0 = 0; c0 < BT && t * BT + c0 < a.T; c0 += 16) {
          uint32_t v[16];
          __syncwarp();
          tmem_ld16(acc + c0, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (t * BT + c0 + c >= a.T) break;
            const int live = min(BT, a.T - t * BT);
            const int to = ((c0 + c + 1) * ranks - 1) / live;  // the rank whose slice holds the token
            const int lo = to * live / ranks, n = (to + 1) * live / ranks - lo;
            store_remote(base + C::kSmemJoin + ((rank * n + c0 + c - lo) * kM + row) * 4, to, __uint_as_float(v[c]));
          }
        }
        cluster_arrive();
        cluster_wait();
        const int live = min(BT, a.T - t * BT), lo = rank * live / ranks, n = (rank + 1) * live / ranks - lo;
        const float* const join = reinterpret_cast<const float*>(smem + C::kSmemJoin) + row;
        for (int c = 0; c < n; ++c) {
          float v = join[c * kM];
          for (int r = 1; r < ranks; ++r) v += join[(r * n + c) * kM];
          finish<1>(a, bias, feature, t * BT + lo + c, &v);
        }
      } else {
        for (int c0 = 0; c0 < BT && t * BT + c0 < a.T; c0 += 16) {
          uint32_t v[16];
          __syncwarp();
          tmem_ld16(acc + c0, v);
          float p[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) p[c] = __uint_as_float(v[c]);
          finish<16>(a, bias, feature, t * BT + c0, p);
        }
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

template <class C>
cudaError_t launch_t(LinearArgs a, int split, cudaStream_t s) {
  auto kern = linear_kernel<C>;
  static PerDevice opted;
  cudaError_t err = cudaSuccess;
  opted([&](int) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    return err == cudaSuccess ? 1 : 0;
  });
  if (err != cudaSuccess) return err;
  CUtensorMap wm, xm;
  if (!make_map(&wm, a.x_dtype, a.w, a.N, a.K, a.w_stride, kM) || !make_map(&xm, a.x_dtype, a.x, a.T, a.K, a.x_stride, C::BT))
    return cudaErrorInvalidValue;
  a.split = split;
  const int64_t tiles = (int64_t)((a.N + kM - 1) / kM) * ((a.T + C::BT - 1) / C::BT);
  const int64_t grid = C::kSplit ? tiles * split : std::min<int64_t>(tiles, (int64_t)C::kPerSm * num_sms());
  note_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = C::kSplit ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, wm, xm);
}
template <int BT>
cudaError_t launch_tokens(const LinearArgs& a, int split, cudaStream_t s) {
  return split > 1 ? launch_t<Cfg<BT, true>>(a, split, s) : launch_t<Cfg<BT, false>>(a, 1, s);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  if (a.T == 0 || a.N == 0) return cudaSuccess;
  const int sms = num_sms(), blocks = (a.K + kK - 1) / kK;
  int best_bt = 256, best_split = 1;
  double best = 1e30;
  for (int bt = 16; bt <= 256; bt *= 2) {
    const int64_t tiles = (int64_t)((a.N + kM - 1) / kM) * ((a.T + bt - 1) / bt);
    const int room = (bt <= 32 ? 2 : 1) * sms;
    for (int split = 1; split <= (bt <= 128 ? 8 : 1) && split <= std::max(1, blocks / 2); ++split) {
      if (split > 1 && tiles * split > room) break;
      const double waves = std::ceil((double)tiles * split / room);
      // cycles: a stage's copies or its products; an accumulator's way out
      const double stage = std::max(2.0 * bt, (kW + bt * 128.0) / (bt <= 32 ? 24.0 : 48.0));
      const double cost = waves * stage * ((blocks + split - 1) / split) + 2500 + 12.0 * std::min(bt, a.T) + (split > 1 ? 1500 : 0);
      if (cost < best) best = cost, best_bt = bt, best_split = split;
    }
  }
  switch (best_bt) {
    case 16: return launch_tokens<16>(a, best_split, s);
    case 32: return launch_tokens<32>(a, best_split, s);
    case 64: return launch_tokens<64>(a, best_split, s);
    case 128: return launch_tokens<128>(a, best_split, s);
    default: return launch_t<Cfg<256, false>>(a, 1, s);
  }
}

}  // namespace moe
