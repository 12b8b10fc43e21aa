// C ABI of the decoder-block operators around the experts: argument
// validation and dispatch.  As in the layer's entry points, everything is
// checked on the host before a launch.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "moe_internal.h"

namespace moe {
namespace {

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int done(cudaError_t e) { return record_error(e) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool dtype_ok(int dt) { return dt == MOE_DT_F32 || dt == MOE_DT_BF16 || dt == MOE_DT_F16; }
int dtype_size(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }
// rows of `stride` elements of type dt all start on 16-byte boundaries
bool rows16(const void* p, int64_t stride, int dt, int64_t T) {
  return !p || (aligned_to(p, 16) && (T <= 1 || stride * dtype_size(dt) % 16 == 0));
}

// sizes of a cache (eight: of 8-bit codes); MOE_OK or why not
int kv_desc_check(const moe_kv_desc* kv, bool eight = false) {
  if (!kv) return MOE_ERR_INVALID_ARG;
  if (eight ? kv->dtype != MOE_DT_E4M3 && kv->dtype != MOE_DT_INT8 : kv->dtype != MOE_DT_BF16 && kv->dtype != MOE_DT_F16)
    return MOE_ERR_UNSUPPORTED;
  if (kv->D < 8 || kv->D > 256 || kv->D % 8 || kv->Hkv < 1 || kv->Hkv > 1024) return MOE_ERR_UNSUPPORTED;
  if (kv->n_seqs < 1 || kv->n_seqs > MOE_MAX_SEQS) return MOE_ERR_UNSUPPORTED;
  if (kv->page_size < 1 || kv->num_pages < 1 || kv->max_pages < 1 || kv->reserved != 0) return MOE_ERR_INVALID_ARG;
  if ((int64_t)kv->max_pages * kv->page_size > (int64_t)INT32_MAX - 1024) return MOE_ERR_UNSUPPORTED;
  if (kv->table_stride < kv->max_pages && kv->n_seqs > 1) return MOE_ERR_INVALID_ARG;
  const int64_t st[6] = {kv->k_page_stride, kv->k_row_stride, kv->k_head_stride,
                         kv->v_page_stride, kv->v_row_stride, kv->v_head_stride};
  for (int64_t v : st)
    if (v < 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
// a stride over a dimension of one entry is never used: whatever it holds, it counts as 0
moe_kv_desc tidy(moe_kv_desc kv) {
  if (kv.num_pages == 1) kv.k_page_stride = kv.v_page_stride = 0;
  if (kv.page_size == 1) kv.k_row_stride = kv.v_row_stride = 0;
  if (kv.Hkv == 1) kv.k_head_stride = kv.v_head_stride = 0;
  return kv;
}
// the scales of an 8-bit cache
int scales_check(const moe_kv_scales* sc) {
  if (!sc || !sc->k || !sc->v || !aligned_to(sc->k, 4) || !aligned_to(sc->v, 4)) return MOE_ERR_INVALID_ARG;
  const int64_t st[6] = {sc->k_page_stride, sc->k_row_stride, sc->k_head_stride,
                         sc->v_page_stride, sc->v_row_stride, sc->v_head_stride};
  for (int64_t v : st)
    if (v < 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
// all strides of a cache's codes are multiples of n bytes
bool code_strides(const moe_kv_desc& kv, int n) {
  return kv.k_page_stride % n == 0 && kv.k_row_stride % n == 0 && kv.k_head_stride % n == 0 &&
         kv.v_page_stride % n == 0 && kv.v_row_stride % n == 0 && kv.v_head_stride % n == 0;
}
struct Dim {
  int64_t n, stride;
};
// Whether pieces of `piece` elements over some dimensions share none: by rising stride, each dimension's entries lie behind
// all of the dimensions before it.
template <int N>
bool apart(Dim (&d)[N], int64_t piece) {
  std::sort(d, d + N, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  __int128 span = piece;
  for (const Dim& x : d) {
    if (x.n <= 1) continue;
    if (x.stride < span) return false;
    span += (__int128)(x.n - 1) * x.stride;
  }
  return true;
}
// the entries of a cache that is written: (page, row, head)
bool entries_apart(const moe_kv_desc& kv, int64_t page, int64_t row, int64_t head, int64_t piece) {
  Dim d[3] = {{kv.num_pages, page}, {kv.page_size, row}, {kv.Hkv, head}};
  return apart(d, piece);
}
// An array of n rows of `bytes` bytes, `stride` bytes apart.
struct Rows {
  const void* p;
  int64_t n, bytes, stride;
};
// Whether two arrays share a byte.  Rows that lie among one another are told apart where the strides are the same, or one
// array has a single row; others whose spans overlap count as shared.
bool share(const Rows& a, const Rows& b) {
  using Wide = __int128;
  if (!a.p || !b.p || a.n < 1 || b.n < 1) return false;
  const Wide at = (Wide)reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p);  // b's first row from a's
  if (at >= (Wide)(a.n - 1) * a.stride + a.bytes || -at >= (Wide)(b.n - 1) * b.stride + b.bytes) return false;
  if (a.n > 1 && b.n > 1 && a.stride != b.stride) return true;
  const Wide s = a.n > 1 ? a.stride : b.stride;
  if ((a.n == 1 && b.n == 1) || s == 0) return true;
  // row j of b from row i of a: at + (j - i) s, between -b.bytes and a.bytes where they meet
  const auto down = [s](Wide x) { return x >= 0 ? x / s : -((-x + s - 1) / s); };
  const Wide least = down(-b.bytes - at) + 1, most = down(a.bytes - 1 - at);  // of j - i
  return std::max<Wide>(least, 1 - a.n) <= std::min<Wide>(most, b.n - 1);
}
bool kv_strides16(const moe_kv_desc& kv) {
  return kv.k_page_stride % 8 == 0 && kv.k_row_stride % 8 == 0 && kv.k_head_stride % 8 == 0 &&
         kv.v_page_stride % 8 == 0 && kv.v_row_stride % 8 == 0 && kv.v_head_stride % 8 == 0;
}

// moe_linear with its plan (tokens 0: by cost)
int linear(const void* x, int32_t x_dtype, int64_t x_stride, const void* w, int64_t w_stride, const float* bias,
           int32_t act, const void* residual, int32_t r_dtype, int64_t r_stride, void* out, int32_t o_dtype,
           int64_t o_stride, int32_t T, int32_t N, int32_t K, int32_t* status, void* stream, LinearPlan plan) {
  if (!residual) r_dtype = x_dtype;
  if (T < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
  if ((r_dtype != x_dtype && r_dtype != MOE_DT_F32) || (o_dtype != x_dtype && o_dtype != MOE_DT_F32)) return MOE_ERR_UNSUPPORTED;
  if (act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH || K % 8) return MOE_ERR_UNSUPPORTED;
  // tiles and rows are 32-bit numbers
  if (((int64_t)N / 128 + 1) * ((int64_t)T / 16 + 1) > 1 << 30 || T > INT32_MAX - 1024 || N > INT32_MAX - 1024 || K > INT32_MAX - 1024)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w || !out) return MOE_ERR_INVALID_ARG;
  if (T > 1 && (x_stride < K || o_stride < N || (residual && r_stride < N))) return MOE_ERR_INVALID_ARG;
  if (N > 1 && w_stride < K) return MOE_ERR_INVALID_ARG;
  if (T == 1) x_stride = r_stride = o_stride = 0;
  if (N == 1) w_stride = 0;
  if (x_stride % 8 || w_stride % 8 || x_stride >= (int64_t)1 << 39 || w_stride >= (int64_t)1 << 39) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(bias, 4) || !aligned_to(residual, dtype_size(r_dtype)) ||
      !aligned_to(out, dtype_size(o_dtype)) || !aligned_to(status, 4))
    return MOE_ERR_INVALID_ARG;
  // tiles are written while others are read; a residual's element is read by the thread that writes its place
  const auto rows = [](const void* p, int64_t n, int64_t cols, int64_t stride, int size) {
    return Rows{p, n, cols * size, stride * size};
  };
  const Rows to = rows(out, T, N, o_stride, dtype_size(o_dtype));
  const bool in_place = residual == out && r_dtype == o_dtype && r_stride == o_stride;
  if (share(to, rows(x, T, K, x_stride, 2)) || share(to, rows(w, N, K, w_stride, 2)) || share(to, rows(bias, 1, N, 0, 4)) ||
      (!in_place && share(to, rows(residual, T, N, r_stride, dtype_size(r_dtype)))) || share(to, rows(status, 1, 1, 0, 4)))
    return MOE_ERR_INVALID_ARG;
  LinearArgs a{};
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.x_stride = x_stride;
  a.w_stride = w_stride;
  a.r_stride = r_stride;
  a.o_stride = o_stride;
  a.x_dtype = x_dtype;
  a.r_dtype = r_dtype;
  a.o_dtype = o_dtype;
  a.act = act;
  a.T = T;
  a.N = N;
  a.K = K;
  a.status = status;
  return done(launch_linear(a, plan, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_add_rmsnorm(const void* x, int32_t x_dtype, int64_t x_stride, const void* residual, int32_t r_dtype,
                    int64_t r_stride, const void* weight, int32_t w_dtype, float weight_offset, float eps, int64_t T,
                    int32_t H, void* sum_out, int64_t sum_stride, void* y, int32_t y_dtype, int64_t y_stride,
                    int32_t q_fmt, void* q, float* d, int16_t* bsum16, void* stream) {
  if (!residual) r_dtype = x_dtype;
  if (!y) y_dtype = x_dtype;
  if (T < 0 || H < 1 || !(eps >= 0.0f) || std::isnan(weight_offset)) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(x_dtype) || !dtype_ok(r_dtype) || !dtype_ok(w_dtype) || !dtype_ok(y_dtype)) return MOE_ERR_UNSUPPORTED;
  if (r_dtype != x_dtype && r_dtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
  if (q_fmt < MOE_NORM_Q_NONE || q_fmt > MOE_NORM_Q_INT8_ROW) return MOE_ERR_UNSUPPORTED;
  if (H > MOE_MAX_DIM || T > INT32_MAX || (q_fmt == MOE_NORM_Q_Q8K && H % 256)) return MOE_ERR_UNSUPPORTED;
  if (bsum16 && q_fmt != MOE_NORM_Q_Q8K) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !weight || (!sum_out && !y && q_fmt == MOE_NORM_Q_NONE)) return MOE_ERR_INVALID_ARG;
  if (q_fmt != MOE_NORM_Q_NONE && (!q || !d)) return MOE_ERR_INVALID_ARG;
  if (T > 1 && (x_stride < H || (residual && r_stride < H) || (sum_out && sum_stride < H) || (y && y_stride < H)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned_to(x, dtype_size(x_dtype)) || !aligned_to(residual, dtype_size(r_dtype)) ||
      !aligned_to(weight, dtype_size(w_dtype)) || !aligned_to(sum_out, dtype_size(r_dtype)) ||
      !aligned_to(y, dtype_size(y_dtype)) || !aligned_to(d, 4) || !aligned_to(bsum16, 2))
    return MOE_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.w = weight;
  a.sum_out = sum_out;
  a.y = y;
  a.q = q;
  a.d = d;
  a.bsum16 = bsum16;
  a.x_dtype = x_dtype;
  a.r_dtype = r_dtype;
  a.w_dtype = w_dtype;
  a.y_dtype = y_dtype;
  a.q_fmt = q_fmt;
  a.x_stride = x_stride;
  a.r_stride = r_stride;
  a.sum_stride = sum_stride;
  a.y_stride = y_stride;
  a.T = T;
  a.H = H;
  a.eps = eps;
  a.w_offset = weight_offset;
  a.wide = H % 8 == 0 && rows16(x, x_stride, x_dtype, T) && rows16(residual, r_stride, r_dtype, T) &&
           rows16(sum_out, sum_stride, r_dtype, T) && rows16(y, y_stride, y_dtype, T) && aligned_to(weight, 16) &&
           aligned_to(q, 8);
  return done(launch_add_rmsnorm(a, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_route_grouped(const void* logits, int32_t dtype, int64_t stride, const float* bias, int32_t T, int32_t E,
                      int32_t k, int32_t route, int32_t n_group, int32_t topk_group, int32_t group_score,
                      int32_t renorm, float scale, int32_t* ids, float* gates, void* stream) {
  if (T < 0 || k < 1 || E < 1 || n_group < 1 || topk_group < 1) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || E > MOE_MAX_EXPERTS || k > MOE_MAX_TOPK || k > E) return MOE_ERR_UNSUPPORTED;
  if (route != MOE_ROUTE_SOFTMAX && route != MOE_ROUTE_SIGMOID) return MOE_ERR_UNSUPPORTED;
  if (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2) return MOE_ERR_UNSUPPORTED;
  if (n_group > 32 || E % n_group || topk_group > n_group || (int64_t)topk_group * (E / n_group) < k)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !ids || !gates || (T > 1 && stride < E)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(logits, dtype_size(dtype)) || !aligned_to(bias, 4) || !aligned_to(ids, 4) || !aligned_to(gates, 4))
    return MOE_ERR_INVALID_ARG;
  RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.gates = gates;
  a.stride = stride;
  a.dtype = dtype;
  a.T = T;
  a.E = E;
  a.k = k;
  a.route = route;
  a.n_group = topk_group == n_group ? 1 : n_group;  // every group kept: no groups
  a.topk_group = a.n_group == 1 ? 1 : topk_group;
  a.group_score = group_score;
  a.renorm = renorm;
  a.scale = scale;
  return done(launch_route_grouped(a, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_kv_append(const moe_kv_desc* kv, const void* k, int64_t k_stride, int64_t k_head_stride, const void* v,
                  int64_t v_stride, int64_t v_head_stride, void* k_cache, void* v_cache, const int32_t* page_table,
                  const int32_t* cu_q, const int32_t* kv_len, int32_t T, void* ws, size_t ws_bytes, void* stream) {
  const int why = kv_desc_check(kv);
  if (why != MOE_OK) return why;
  if (T < 0 || k_stride < 0 || k_head_stride < 0 || v_stride < 0 || v_head_stride < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!k || !v || !k_cache || !v_cache || !page_table || !cu_q || !kv_len || !ws) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < 16) return MOE_ERR_WORKSPACE;
  if (!aligned_to(k, 2) || !aligned_to(v, 2) || !aligned_to(k_cache, 2) || !aligned_to(v_cache, 2) ||
      !aligned_to(page_table, 4) || !aligned_to(cu_q, 4) || !aligned_to(kv_len, 4) || !aligned_to(ws, 16))
    return MOE_ERR_INVALID_ARG;
  KvAppendArgs a{};
  a.kv = tidy(*kv);
  if (T == 1) k_stride = v_stride = 0;
  if (kv->Hkv == 1) k_head_stride = v_head_stride = 0;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.k_head_stride = k_head_stride;
  a.v_stride = v_stride;
  a.v_head_stride = v_head_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.table = page_table;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.T = T;
  a.status = static_cast<int*>(ws);
  a.wide = kv_strides16(a.kv) && k_stride % 8 == 0 && k_head_stride % 8 == 0 && v_stride % 8 == 0 &&
           v_head_stride % 8 == 0 && aligned_to(k, 16) && aligned_to(v, 16) && aligned_to(k_cache, 16) &&
           aligned_to(v_cache, 16);
  return done(launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_kv_append_q8(const moe_kv_desc* kv, const moe_kv_scales* scales, int32_t x_dtype, const void* k,
                     int64_t k_stride, int64_t k_head_stride, const void* v, int64_t v_stride, int64_t v_head_stride,
                     void* k_cache, void* v_cache, const int32_t* page_table, const int32_t* cu_q,
                     const int32_t* kv_len, int32_t T, void* ws, size_t ws_bytes, void* stream) {
  const int why = kv_desc_check(kv, true);
  if (why != MOE_OK) return why;
  if (x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
  if (T < 0 || k_stride < 0 || k_head_stride < 0 || v_stride < 0 || v_head_stride < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!k || !v || !k_cache || !v_cache || !page_table || !cu_q || !kv_len || !ws) return MOE_ERR_INVALID_ARG;
  if (scales_check(scales) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < 16) return MOE_ERR_WORKSPACE;
  if (!aligned_to(k, 2) || !aligned_to(v, 2) || !aligned_to(page_table, 4) || !aligned_to(cu_q, 4) ||
      !aligned_to(kv_len, 4) || !aligned_to(ws, 16))
    return MOE_ERR_INVALID_ARG;
  // a code beside another entry's scale would be neither's (a cache that is only read may repeat entries)
  if (!entries_apart(*kv, kv->k_page_stride, kv->k_row_stride, kv->k_head_stride, kv->D) ||
      !entries_apart(*kv, kv->v_page_stride, kv->v_row_stride, kv->v_head_stride, kv->D) ||
      !entries_apart(*kv, scales->k_page_stride, scales->k_row_stride, scales->k_head_stride, 1) ||
      !entries_apart(*kv, scales->v_page_stride, scales->v_row_stride, scales->v_head_stride, 1))
    return MOE_ERR_INVALID_ARG;
  KvAppendQ8Args g{};
  KvAppendArgs& a = g.a;
  a.kv = tidy(*kv);
  if (T == 1) k_stride = v_stride = 0;
  if (kv->Hkv == 1) k_head_stride = v_head_stride = 0;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.k_head_stride = k_head_stride;
  a.v_stride = v_stride;
  a.v_head_stride = v_head_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.table = page_table;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.T = T;
  a.status = static_cast<int*>(ws);
  a.wide = code_strides(a.kv, 8) && k_stride % 8 == 0 && k_head_stride % 8 == 0 && v_stride % 8 == 0 &&
           v_head_stride % 8 == 0 && aligned_to(k, 16) && aligned_to(v, 16) && aligned_to(k_cache, 8) &&
           aligned_to(v_cache, 8);
  g.sc = *scales;
  g.x_dtype = x_dtype;
  return done(launch_kv_append_q8(g, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_kv_read_q8(const moe_kv_desc* kv, const moe_kv_scales* scales, const void* k_cache, const void* v_cache,
                   const int32_t* page_table, const int32_t* kv_len, const int32_t* first, int32_t n_rows,
                   int32_t out_dtype, void* k_out, int64_t k_stride, int64_t k_head_stride, void* v_out,
                   int64_t v_stride, int64_t v_head_stride, void* ws, size_t ws_bytes, void* stream) {
  const int why = kv_desc_check(kv, true);
  if (why != MOE_OK) return why;
  if (!dtype_ok(out_dtype)) return MOE_ERR_UNSUPPORTED;
  if (n_rows < 0 || k_stride < 0 || k_head_stride < 0 || v_stride < 0 || v_head_stride < 0) return MOE_ERR_INVALID_ARG;
  // without rows the lengths alone are looked at: no key has a place
  if (n_rows == 0 && (!kv_len || !first || !ws)) return MOE_OK;
  if (!kv_len || !first || !ws) return MOE_ERR_INVALID_ARG;
  if (n_rows > 0 && (!k_cache || !v_cache || !page_table || !k_out || !v_out || scales_check(scales) != MOE_OK))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < 16) return MOE_ERR_WORKSPACE;
  const int es = dtype_size(out_dtype);
  if (!aligned_to(page_table, 4) || !aligned_to(kv_len, 4) || !aligned_to(first, 4) || !aligned_to(ws, 16) ||
      !aligned_to(k_out, es) || !aligned_to(v_out, es))
    return MOE_ERR_INVALID_ARG;
  if (kv->Hkv == 1) k_head_stride = v_head_stride = 0;
  if (n_rows == 1) k_stride = v_stride = 0;
  // rows that overlap would be written in no order
  Dim ko[2] = {{n_rows, k_stride}, {kv->Hkv, k_head_stride}}, vo[2] = {{n_rows, v_stride}, {kv->Hkv, v_head_stride}};
  if (n_rows > 0 && (!apart(ko, kv->D) || !apart(vo, kv->D))) return MOE_ERR_INVALID_ARG;
  KvReadQ8Args a{};
  a.kv = tidy(*kv);
  if (scales) a.sc = *scales;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.table = page_table;
  a.kv_len = kv_len;
  a.first = first;
  a.rows = n_rows;
  a.out_dtype = out_dtype;
  a.k_out = k_out;
  a.v_out = v_out;
  a.k_stride = k_stride;
  a.k_head_stride = k_head_stride;
  a.v_stride = v_stride;
  a.v_head_stride = v_head_stride;
  a.status = static_cast<int*>(ws);
  const int per = 16 / es;
  a.wide = kv->D % 16 == 0 && code_strides(a.kv, 16) && aligned_to(k_cache, 16) && aligned_to(v_cache, 16) &&
           k_stride % per == 0 && k_head_stride % per == 0 && v_stride % per == 0 && v_head_stride % per == 0 &&
           aligned_to(k_out, 16) && aligned_to(v_out, 16);
  return done(launch_kv_read_q8(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_paged_attention_workspace_size(int32_t Hq, int32_t Hkv, int32_t D) {
  if (Hkv < 1 || Hkv > 1024 || Hq < 1 || Hq > 1024 || Hq % Hkv || D < 8 || D > 256 || D % 8) return 0;
  return attn_workspace(Hq, Hkv, D);
}

int moe_paged_attention(const moe_kv_desc* kv, const void* q, int64_t q_stride, int64_t q_head_stride, int32_t Hq,
                        int32_t T, const void* k_cache, const void* v_cache, const int32_t* page_table,
                        const int32_t* cu_q, const int32_t* kv_len, float scale, int32_t window, void* out,
                        int64_t o_stride, int64_t o_head_stride, float* lse, void* ws, size_t ws_bytes, void* stream) {
  const int why = kv_desc_check(kv);
  if (why != MOE_OK) return why;
  if (T < 0 || Hq < 1 || window < 0 || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (Hq > 1024 || Hq % kv->Hkv || (int64_t)T * Hq > INT32_MAX - 1024) return MOE_ERR_UNSUPPORTED;
  if (q_stride < 0 || q_head_stride < 0 || o_stride < 0 || o_head_stride < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!q || !k_cache || !v_cache || !page_table || !cu_q || !kv_len || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(out, 16) ||
      !aligned_to(page_table, 4) || !aligned_to(cu_q, 4) || !aligned_to(kv_len, 4) || !aligned_to(lse, 4) ||
      !aligned_to(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (T == 1) q_stride = o_stride = 0;
  if (Hq == 1) q_head_stride = o_head_stride = 0;
  if (!kv_strides16(tidy(*kv)) || q_stride % 8 || q_head_stride % 8 || o_stride % 8 || o_head_stride % 8)
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < attn_workspace(Hq, kv->Hkv, kv->D)) return MOE_ERR_WORKSPACE;
  if (attn_tensor_core(*kv) && !attn_units_fit(*kv, Hq, T)) return MOE_ERR_UNSUPPORTED;
  AttnArgs a{};
  a.kv = tidy(*kv);
  a.q = q;
  a.q_stride = q_stride;
  a.q_head_stride = q_head_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.table = page_table;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.Hq = Hq;
  a.T = T;
  a.window = window;
  a.scale = scale;
  a.out = out;
  a.o_stride = o_stride;
  a.o_head_stride = o_head_stride;
  a.lse = lse;
  a.ws = static_cast<char*>(ws);
  a.status = static_cast<int*>(ws);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return done(attn_tensor_core(a.kv) ? launch_attn(a, s) : launch_attn_general(a, s));
}

size_t moe_paged_attention_q8_workspace_size(int32_t Hq, int32_t Hkv, int32_t D) {
  if (Hkv < 1 || Hkv > 1024 || Hq < 1 || Hq > 1024 || Hq % Hkv || D < 8 || D > 256 || D % 8) return 0;
  return attn_q8_workspace(Hq, Hkv, D);
}

int moe_paged_attention_q8(const moe_kv_desc* kv, const moe_kv_scales* scales, int32_t x_dtype, const void* q,
                           int64_t q_stride, int64_t q_head_stride, int32_t Hq, int32_t T, const void* k_cache,
                           const void* v_cache, const int32_t* page_table, const int32_t* cu_q, const int32_t* kv_len,
                           float scale, int32_t window, void* out, int64_t o_stride, int64_t o_head_stride, float* lse,
                           void* ws, size_t ws_bytes, void* stream) {
  const int why = kv_desc_check(kv, true);
  if (why != MOE_OK) return why;
  if (x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
  if (T < 0 || Hq < 1 || window < 0 || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (Hq > 1024 || Hq % kv->Hkv || (int64_t)T * Hq > INT32_MAX - 1024) return MOE_ERR_UNSUPPORTED;
  if (q_stride < 0 || q_head_stride < 0 || o_stride < 0 || o_head_stride < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!q || !k_cache || !v_cache || !page_table || !cu_q || !kv_len || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (scales_check(scales) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 8) || !aligned_to(v_cache, 8) || !aligned_to(out, 16) ||
      !aligned_to(page_table, 4) || !aligned_to(cu_q, 4) || !aligned_to(kv_len, 4) || !aligned_to(lse, 4) ||
      !aligned_to(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (T == 1) q_stride = o_stride = 0;
  if (Hq == 1) q_head_stride = o_head_stride = 0;
  const moe_kv_desc d = tidy(*kv);
  if (!code_strides(d, 8) || q_stride % 8 || q_head_stride % 8 || o_stride % 8 || o_head_stride % 8)
    return MOE_ERR_INVALID_ARG;
  Dim o[2] = {{T, o_stride}, {Hq, o_head_stride}};
  if (!apart(o, kv->D)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < attn_q8_workspace(Hq, kv->Hkv, kv->D)) return MOE_ERR_WORKSPACE;
  AttnQ8Args g{};
  AttnArgs& a = g.a;
  a.kv = d;
  a.q = q;
  a.q_stride = q_stride;
  a.q_head_stride = q_head_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.table = page_table;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.Hq = Hq;
  a.T = T;
  a.window = window;
  a.scale = scale;
  a.out = out;
  a.o_stride = o_stride;
  a.o_head_stride = o_head_stride;
  a.lse = lse;
  a.ws = static_cast<char*>(ws);
  a.status = static_cast<int*>(ws);
  g.sc = *scales;
  g.x_dtype = x_dtype;
  g.G = Hq / kv->Hkv;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (attn_q8_tensor_core(g) && !attn_q8_fits(g)) return MOE_ERR_UNSUPPORTED;
  return done(attn_q8_tensor_core(g) ? launch_attn_q8(g, s) : launch_attn_q8_general(g, s));
}

int moe_linear(const void* x, int32_t x_dtype, int64_t x_stride, const void* w, int64_t w_stride, const float* bias,
               int32_t act, const void* residual, int32_t r_dtype, int64_t r_stride, void* out, int32_t o_dtype,
               int64_t o_stride, int32_t T, int32_t N, int32_t K, int32_t* status, void* stream) {
  return linear(x, x_dtype, x_stride, w, w_stride, bias, act, residual, r_dtype, r_stride, out, o_dtype, o_stride, T, N, K, status,
                stream, LinearPlan{0, 0});
}

int moe_debug_linear(const void* x, int32_t x_dtype, int64_t x_stride, const void* w, int64_t w_stride, const float* bias,
                     int32_t act, const void* residual, int32_t r_dtype, int64_t r_stride, void* out, int32_t o_dtype,
                     int64_t o_stride, int32_t T, int32_t N, int32_t K, int32_t tokens, int32_t ctas, int32_t* status,
                     void* stream) {
  if (!linear_plan_ok(LinearPlan{tokens, ctas}, T, N, K)) return MOE_ERR_UNSUPPORTED;
  return linear(x, x_dtype, x_stride, w, w_stride, bias, act, residual, r_dtype, r_stride, out, o_dtype, o_stride, T, N, K, status,
                stream, LinearPlan{tokens, ctas});
}

}  // extern "C"
