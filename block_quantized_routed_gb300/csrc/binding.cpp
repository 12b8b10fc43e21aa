// The binding of the decoder-block operators: checks tensors and marshals
// their pointers, sizes and strides into the C ABI.
//
// A decode step calls these operators many times with little work in each.
// Through ctypes a call of twenty arguments costs about 10 us of host time, as
// long as several of the kernels take; here it is a few hundred nanoseconds
// before the launch.  Nothing is computed and nothing is kept between calls.
#include <Python.h>

#include <initializer_list>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_q8k.h"

namespace {

PyObject* g_raise = nullptr;  // python callable (status, text) that raises MoeError

struct Refused {
  int status;
  std::string text;
};
[[noreturn]] void refuse(int status, const std::string& text) { throw Refused{status, text}; }
void need(bool ok, const char* text) {
  if (!ok) refuse(MOE_ERR_INVALID_ARG, text);
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(MOE_ERR_INVALID_ARG, std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw std::runtime_error("");
  return v;
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::runtime_error("");
  return v;
}
int32_t int32(PyObject* o, const char* what) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(MOE_ERR_INVALID_ARG, std::string(what) + " is out of range");
  return (int32_t)v;
}
int dtype(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MOE_DT_F32;
    case at::kBFloat16: return MOE_DT_BF16;
    case at::kHalf: return MOE_DT_F16;
    default: refuse(MOE_ERR_UNSUPPORTED, "element type must be float32, bfloat16 or float16");
  }
}
void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
// row stride of a [T, H] tensor with contiguous rows
int64_t rows(const at::Tensor& t, int64_t T, int64_t H, const char* text) {
  need(t.dim() == 2 && t.size(0) == T && t.size(1) == H && (t.stride(1) == 1 || H == 1), text);
  return t.stride(0);
}
void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw std::runtime_error("");
  const unsigned long long v = PyLong_AsUnsignedLongLong(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) throw std::runtime_error("");
  return reinterpret_cast<void*>(v);
}
// every tensor of a call (null: not given) on the current device: a kernel takes them as bare pointers
void on_device(std::initializer_list<const at::Tensor*> ts) {
  int dev = -1;
  for (const at::Tensor* t : ts) {
    if (!t) continue;
    need(t->is_cuda(), "every tensor must be on the GPU");
    need(dev < 0 || t->get_device() == dev, "all tensors must be on one device");
    dev = t->get_device();
  }
  need(dev < 0 || dev == c10::cuda::current_device(), "the tensors' device must be the current one");
}
size_t bytes_of(const at::Tensor& t) { return (size_t)t.numel() * t.element_size(); }

template <typename F>
PyObject* guarded(const char* where, F f) {
  int status;
  std::string text = where;
  try {
    status = f();
  } catch (const Refused& r) {
    status = r.status;
    text += ": " + r.text;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  if (status == MOE_OK) Py_RETURN_NONE;
  PyObject* r = PyObject_CallFunction(g_raise, "is", status, text.c_str());
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, text.c_str());
  return nullptr;
}
bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// x, weight, eps, residual, sum_out, y, q_fmt, q, d, bsum16, weight_offset, stream
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 12)) return nullptr;
  return guarded("moe_add_rmsnorm", [&] {
    const at::Tensor& x = tensor(a[0], "x");
    need(x.dim() == 2, "x must be [T, H]");
    const int64_t T = x.size(0), H = x.size(1);
    need(H <= INT32_MAX, "H is out of range");
    const int64_t xs = rows(x, T, H, "x must have contiguous rows");
    const int xt = dtype(x);
    const at::Tensor& w = tensor(a[1], "weight");
    need(w.dim() == 1 && w.size(0) == H && w.is_contiguous(), "weight must be [H]");
    const at::Tensor *res = maybe(a[3], "residual"), *sum = maybe(a[4], "sum_out"), *y = maybe(a[5], "y");
    const at::Tensor *q = maybe(a[7], "q"), *d = maybe(a[8], "d"), *bs = maybe(a[9], "bsum16");
    int64_t rs = 0, ss = 0, ys = 0;
    int rt = 0, yt = 0;
    if (res) rs = rows(*res, T, H, "residual must be [T, H] with contiguous rows"), rt = dtype(*res);
    if (sum) {
      ss = rows(*sum, T, H, "sum_out must be [T, H] with contiguous rows");
      need(dtype(*sum) == (res ? rt : xt), "sum_out must have the residual's type");
    }
    if (y) ys = rows(*y, T, H, "y must be [T, H] with contiguous rows"), yt = dtype(*y);
    const int32_t fmt = int32(a[6], "q_fmt");
    if (fmt != MOE_NORM_Q_NONE) {
      need(q && d, "q_fmt needs q and d");
      need(q->dim() == 2 && q->size(0) == T && q->size(1) == H && q->element_size() == 1 && q->is_contiguous(),
           "q must be [T, H] of 8 bits");
      const int64_t g = fmt == MOE_NORM_Q_Q8K ? 256 : fmt == MOE_NORM_Q_E4M3_G128 ? 128 : std::max<int64_t>(H, 1);
      need(d->numel() == T * ((H + g - 1) / g) && d->is_contiguous() && d->scalar_type() == at::kFloat,
           "d must hold one fp32 scale per group");
      if (bs)
        need(bs->numel() == T * (H / 16) && bs->scalar_type() == at::kShort && bs->is_contiguous(),
             "bsum16 must be int16 [T, H/16]");
    } else {
      q = d = bs = nullptr;
    }
    on_device({&x, &w, res, sum, y, q, d, bs});
    return moe_add_rmsnorm(x.data_ptr(), xt, xs, ptr(res), rt, rs, w.data_ptr(), dtype(w), (float)number(a[10]),
                           (float)number(a[2]), T, (int32_t)H, ptr(sum), ss, ptr(y), yt, ys, fmt, ptr(q),
                           static_cast<float*>(ptr(d)), static_cast<int16_t*>(ptr(bs)), stream_of(a[11]));
  });
}

// logits, k, ids, gates, bias, route, n_group, topk_group, group_score, renorm, scale, stream
PyObject* route_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 12)) return nullptr;
  return guarded("moe_route_grouped", [&] {
    const at::Tensor& l = tensor(a[0], "logits");
    need(l.dim() == 2 && l.size(0) <= INT32_MAX && l.size(1) <= INT32_MAX, "logits must be [T, E]");
    const int64_t T = l.size(0), E = l.size(1);
    const int64_t stride = rows(l, T, E, "logits must have contiguous rows");
    const int32_t k = int32(a[1], "k");
    const at::Tensor &ids = tensor(a[2], "ids"), &gates = tensor(a[3], "gates");
    need(ids.dim() == 2 && ids.size(0) == T && ids.size(1) == k && ids.is_contiguous() && ids.scalar_type() == at::kInt,
         "ids must be int32 [T, k]");
    need(gates.dim() == 2 && gates.size(0) == T && gates.size(1) == k && gates.is_contiguous() &&
             gates.scalar_type() == at::kFloat,
         "gates must be fp32 [T, k]");
    const at::Tensor* bias = maybe(a[4], "bias");
    if (bias)
      need(bias->dim() == 1 && bias->size(0) == E && bias->is_contiguous() && bias->scalar_type() == at::kFloat,
           "bias must be fp32 [E]");
    const int renorm = PyObject_IsTrue(a[9]);
    if (renorm < 0) throw std::runtime_error("");
    on_device({&l, &ids, &gates, bias});
    return moe_route_grouped(l.data_ptr(), dtype(l), stride, static_cast<const float*>(ptr(bias)), (int32_t)T,
                             (int32_t)E, k, int32(a[5], "route"), int32(a[6], "n_group"), int32(a[7], "topk_group"),
                             int32(a[8], "group_score"), renorm, (float)number(a[10]),
                             ids.data_ptr<int32_t>(), gates.data_ptr<float>(), stream_of(a[11]));
  });
}

// the cache of k_cache, v_cache, page_table, cu_q, kv_len
moe_kv_desc cache(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, const at::Tensor& cu,
                  const at::Tensor& len) {
  need(k.dim() == 4 && k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type(),
       "caches must be [pages, page_size, Hkv, D] of one type");
  need(k.stride(3) == 1 && v.stride(3) == 1, "a head's elements must be contiguous");
  for (int i = 0; i < 4; ++i) need(k.size(i) <= INT32_MAX, "a cache size is out of range");
  need(table.dim() == 2 && (table.stride(1) == 1 || table.size(1) == 1) && table.scalar_type() == at::kInt,
       "page_table must be int32 [n_seqs, max_pages]");
  const int64_t n = table.size(0);
  need(n < INT32_MAX && table.size(1) <= INT32_MAX, "page_table is too large");
  need(cu.dim() == 1 && cu.size(0) == n + 1 && cu.scalar_type() == at::kInt && cu.is_contiguous(),
       "cu_q must be int32 [n_seqs + 1]");
  need(len.dim() == 1 && len.size(0) == n && len.scalar_type() == at::kInt && len.is_contiguous(),
       "kv_len must be int32 [n_seqs]");
  moe_kv_desc d{};
  d.n_seqs = (int32_t)n;
  d.Hkv = (int32_t)k.size(2);
  d.D = (int32_t)k.size(3);
  d.dtype = dtype(k);
  d.page_size = (int32_t)k.size(1);
  d.num_pages = (int32_t)k.size(0);
  d.max_pages = (int32_t)table.size(1);
  d.table_stride = table.stride(0);
  d.k_page_stride = k.stride(0);
  d.k_row_stride = k.stride(1);
  d.k_head_stride = k.stride(2);
  d.v_page_stride = v.stride(0);
  d.v_row_stride = v.stride(1);
  d.v_head_stride = v.stride(2);
  return d;
}
void heads(const at::Tensor& t, int64_t T, int64_t H, const at::Tensor& like, const char* text) {
  need(t.dim() == 3 && t.size(0) == T && t.size(1) == H && t.size(2) == like.size(3) && t.stride(2) == 1 &&
           t.scalar_type() == like.scalar_type(),
       text);
}

// k, v, k_cache, v_cache, page_table, cu_q, kv_len, ws, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  return guarded("moe_kv_append", [&] {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &kc = tensor(a[2], "k_cache");
    const at::Tensor &vc = tensor(a[3], "v_cache"), &table = tensor(a[4], "page_table"), &cu = tensor(a[5], "cu_q");
    const at::Tensor &len = tensor(a[6], "kv_len"), &ws = tensor(a[7], "ws");
    const moe_kv_desc d = cache(kc, vc, table, cu, len);
    need(k.dim() == 3 && k.size(0) <= INT32_MAX, "k must be [T, Hkv, D] of the cache's type");
    heads(k, k.size(0), d.Hkv, kc, "k must be [T, Hkv, D] of the cache's type");
    heads(v, k.size(0), d.Hkv, kc, "v must be like k");
    need(ws.is_contiguous(), "ws must be contiguous");
    on_device({&k, &v, &kc, &vc, &table, &cu, &len, &ws});
    return moe_kv_append(&d, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
                         kc.data_ptr(), vc.data_ptr(), table.data_ptr<int32_t>(), cu.data_ptr<int32_t>(),
                         len.data_ptr<int32_t>(), (int32_t)k.size(0), ws.data_ptr(), bytes_of(ws), stream_of(a[8]));
  });
}

// q, k_cache, v_cache, page_table, cu_q, kv_len, scale, out, ws, lse, window, stream
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 12)) return nullptr;
  return guarded("moe_paged_attention", [&] {
    const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
    const at::Tensor &table = tensor(a[3], "page_table"), &cu = tensor(a[4], "cu_q"), &len = tensor(a[5], "kv_len");
    const at::Tensor &out = tensor(a[7], "out"), &ws = tensor(a[8], "ws");
    const at::Tensor* lse = maybe(a[9], "lse");
    const moe_kv_desc d = cache(kc, vc, table, cu, len);
    need(q.dim() == 3 && q.size(0) <= INT32_MAX && q.size(1) <= INT32_MAX, "q must be [T, Hq, D] of the cache's type");
    const int64_t T = q.size(0), Hq = q.size(1);
    heads(q, T, Hq, kc, "q must be [T, Hq, D] of the cache's type");
    heads(out, T, Hq, kc, "out must be like q");
    if (lse)
      need(lse->dim() == 2 && lse->size(0) == T && lse->size(1) == Hq && lse->is_contiguous() &&
               lse->scalar_type() == at::kFloat,
           "lse must be fp32 [T, Hq]");
    need(ws.is_contiguous(), "ws must be contiguous");
    on_device({&q, &kc, &vc, &table, &cu, &len, &out, &ws, lse});
    return moe_paged_attention(&d, q.data_ptr(), q.stride(0), q.stride(1), (int32_t)Hq, (int32_t)T, kc.data_ptr(),
                               vc.data_ptr(), table.data_ptr<int32_t>(), cu.data_ptr<int32_t>(),
                               len.data_ptr<int32_t>(), (float)number(a[6]), int32(a[10], "window"), out.data_ptr(),
                               out.stride(0), out.stride(1), static_cast<float*>(ptr(lse)), ws.data_ptr(),
                               bytes_of(ws), stream_of(a[11]));
  });
}

PyObject* on_error(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XDECREF(g_raise);
  g_raise = f;
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"add_rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(add_rmsnorm)), METH_FASTCALL, nullptr},
    {"route_grouped", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route_grouped)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attention)), METH_FASTCALL,
     nullptr},
    {"on_error", on_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "moe_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_moe_binding() { return PyModule_Create(&kModule); }
