// C ABI of the decoder-block operators around the experts: argument
// validation and dispatch.  As in the layer's entry points, everything is
// checked on the host before a launch.
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

// sizes of a cache; MOE_OK or why not
int kv_desc_check(const moe_kv_desc* kv) {
  if (!kv) return MOE_ERR_INVALID_ARG;
  if (kv->dtype != MOE_DT_BF16 && kv->dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
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
bool kv_strides16(const moe_kv_desc& kv) {
  return kv.k_page_stride % 8 == 0 && kv.k_row_stride % 8 == 0 && kv.k_head_stride % 8 == 0 &&
         kv.v_page_stride % 8 == 0 && kv.v_row_stride % 8 == 0 && kv.v_head_stride % 8 == 0;
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

}  // extern "C"
