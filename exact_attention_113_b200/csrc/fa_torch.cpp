// fa_torch.cpp -- compiled binding of the serving entries (include/fa.h) for
// torch tensors.  These calls run for every layer of a decoding step, whose
// kernels take some ten microseconds; the same checks and allocations in
// Python through ctypes cost 15 to 30 of them, here 4 to 8.  Argument
// marshalling only: checks, output allocation, the device and the stream; the
// operators themselves are libfa.so's.
#include <Python.h>

#include <cmath>
#include <cstring>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

namespace {

PyObject *g_error = nullptr;   // binding.FaError(status, where)

// Thrown where a Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject *type, const char *fmt, const char *name = "") {
  PyErr_Format(type, fmt, name);
  throw Raised();
}
[[noreturn]] void bad(const char *fmt, const char *name = "") { raise(PyExc_ValueError, fmt, name); }

// A tensor argument; nullptr for None where that is allowed.
const at::Tensor *tensor(PyObject *o, const char *name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch tensor", name);
  return &THPVariable_Unpack(o);
}

long long integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
int int32(PyObject *o, const char *name) {
  const long long v = integer(o);
  if (v != static_cast<int>(v)) bad("%s is out of range", name);
  return static_cast<int>(v);
}
double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}
int size32(int64_t n, const char *name) {
  if (n > 0x7fffffff) bad("%s is too large", name);
  return static_cast<int>(n);
}

// The device of the first tensor; every other one has to be there.
struct Device {
  c10::DeviceIndex index = -1;
  void on(const at::Tensor *t, const char *name) {
    if (!t) return;
    if (!t->is_cuda() || (index >= 0 && t->get_device() != index))
      bad("%s must be a CUDA tensor on the same device as the others", name);
    index = static_cast<c10::DeviceIndex>(t->get_device());
  }
};

// The call's stream: the given one, which also becomes the current one for the
// call, so that what is allocated here belongs to it (a workspace freed on
// return is then not handed to another stream's kernels while this call's
// still run), or the current one.
struct Stream {
  c10::cuda::OptionalCUDAStreamGuard guard;
  cudaStream_t s;
  Stream(PyObject *handle, c10::DeviceIndex dev) {
    if (handle == Py_None) {
      s = c10::cuda::getCurrentCUDAStream(dev).stream();
    } else {
      s = reinterpret_cast<cudaStream_t>(integer(handle));
      guard.reset_stream(c10::cuda::getStreamFromExternal(s, dev));
    }
  }
};

template <typename F>
void call(const char *where, F &&f) {
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  if (st != FA_OK) {
    PyObject *e = PyObject_CallFunction(g_error, "is", st, where);
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    throw Raised();
  }
}

void vec(const at::Tensor *t, const char *name, at::ScalarType type, int64_t n) {
  if (t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
    bad("%s must be a contiguous vector of the right type and length", name);
}

// A workspace's size is taken from its elements, which have to lie in it.
void workspace(const at::Tensor *t) {
  if (t && !t->is_contiguous()) bad("%s must be contiguous", "workspace");
}

int dtype_of(const at::Tensor *q) {
  if (q->scalar_type() == at::kHalf) return FA_F16;
  if (q->scalar_type() == at::kBFloat16) return FA_BF16;
  raise(PyExc_TypeError, "%sdtype must be float16 or bfloat16");
}

struct Cache {
  int pages, page_size;
  long long sp, st, sh;
};
Cache cache_of(const at::Tensor *k, const at::Tensor *v, int64_t H_kv, int64_t D,
               at::ScalarType type) {
  if (k->dim() != 4 || k->sizes() != v->sizes() || k->size(2) != H_kv || k->size(3) != D)
    bad("%sk_cache, v_cache must be [pages, page_size, H_kv, D]");
  if (k->scalar_type() != type || v->scalar_type() != type)
    raise(PyExc_TypeError, "%sk_cache, v_cache must have q's dtype");
  if (k->strides() != v->strides() || k->stride(3) != 1)
    bad("%sk_cache, v_cache must have the same strides, contiguous along D");
  return {size32(k->size(0), "pages"), size32(k->size(1), "page_size"), k->stride(0), k->stride(1),
          k->stride(2)};
}

struct Table {
  int columns;
  long long stride;
};
Table table_of(const at::Tensor *t, int64_t B) {
  if (t->dim() != 2 || t->scalar_type() != at::kInt || t->size(0) != B ||
      (t->size(1) > 1 && t->stride(1) != 1))
    bad("%sblock_table must be int32 [B, max_pages], contiguous along the pages");
  const int n = size32(t->size(1), "max_pages");
  return {n, B > 1 ? t->stride(0) : (n > 0 ? n : 1)};
}

// [T, H, D] or [B, L, H, D] rows of the given shape.
fa_rows rows_of(const at::Tensor *t, const char *name, at::IntArrayRef shape, at::ScalarType type) {
  const int64_t n = t->dim();
  if (t->sizes() != shape || t->scalar_type() != type || t->stride(n - 1) != 1)
    bad("%s must have q's (k's) shape and dtype, contiguous along D", name);
  return {t->data_ptr(), n == 4 ? t->stride(0) : 0, t->stride(n - 3), t->stride(n - 2)};
}

at::Tensor empty(at::IntArrayRef shape, const at::Tensor *like, at::ScalarType type) {
  return at::empty(shape, like->options().dtype(type).memory_format(c10::nullopt));
}

// n elements of `type` at element `at` of buf's storage, as a tensor of its own
// (a view through the dispatcher takes five times as long).
at::Tensor part(const at::Tensor &buf, at::ScalarType type, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(buf.storage()), buf.key_set(), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "%swrong number of arguments");
}

#define FA_BEGIN HANDLE_TH_ERRORS try {
#define FA_END                     \
  }                                \
  catch (const Raised &) {         \
    return nullptr;                \
  }                                \
  END_HANDLE_TH_ERRORS

// ------------------------------------------------------------------ paged_plan
// (q_lens, ctx_lens, block_table, free_pages, page_size, num_tokens, out | None, stream | None)
PyObject *paged_plan(PyObject *, PyObject *const *a, Py_ssize_t na) {
  FA_BEGIN
  count(na, 8);
  const at::Tensor *q = tensor(a[0], "q_lens"), *ctx = tensor(a[1], "ctx_lens"),
                   *table = tensor(a[2], "block_table"), *free_pages = tensor(a[3], "free_pages");
  if (q->dim() != 1 || free_pages->dim() != 1) bad("%sq_lens and free_pages must be vectors");
  const int B = size32(q->size(0), "q_lens"), n_free = size32(free_pages->size(0), "free_pages");
  const int page_size = int32(a[4], "page_size"), T = int32(a[5], "num_tokens");
  vec(q, "q_lens", at::kInt, B);
  vec(ctx, "ctx_lens", at::kInt, B);
  vec(free_pages, "free_pages", at::kInt, n_free);
  const Table tb = table_of(table, B);
  Device dev;
  dev.on(q, "q_lens");
  dev.on(ctx, "ctx_lens");
  dev.on(table, "block_table");
  dev.on(free_pages, "free_pages");
  if (T < 0) bad("%snum_tokens must be >= 0");
  at::Tensor o[5];   // cu_q, kv_lens, positions, slots, counts
  const int64_t n[5] = {B + 1, B, T, T, 3};
  c10::cuda::CUDAGuard guard(dev.index);
  const Stream stream(a[7], dev.index);
  if (a[6] == Py_None) {
    // one allocation, the 8-byte values first
    const at::Tensor buf = empty({2ll * T + T + 2ll * B + 4}, q, at::kInt);
    o[3] = part(buf, at::kLong, 0, T);
    int64_t at = 2ll * T;
    for (int i : {2, 0, 1, 4}) {
      o[i] = part(buf, at::kInt, at, n[i]);
      at += n[i];
    }
  } else {
    if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 5) bad("%sout must be a PagedPlan");
    static const char *names[5] = {"cu_q", "kv_lens", "positions", "slots", "counts"};
    for (int i = 0; i < 5; ++i) {
      const at::Tensor *t = tensor(PyTuple_GET_ITEM(a[6], i), names[i]);
      vec(t, names[i], i == 3 ? at::kLong : at::kInt, n[i]);
      dev.on(t, names[i]);
      o[i] = *t;
    }
  }
  call("fa_paged_plan", [&] {
    return fa_paged_plan(static_cast<int *>(q->data_ptr()), static_cast<int *>(ctx->data_ptr()),
                         static_cast<int *>(table->data_ptr()), tb.stride,
                         static_cast<int *>(free_pages->data_ptr()), n_free, B, tb.columns,
                         page_size, T, static_cast<int *>(o[0].data_ptr()),
                         static_cast<int *>(o[1].data_ptr()), static_cast<int *>(o[2].data_ptr()),
                         static_cast<long long *>(o[3].data_ptr()),
                         static_cast<int *>(o[4].data_ptr()), stream.s);
  });
  PyObject *r = PyTuple_New(5);
  for (int i = 0; r && i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(o[i])));
  return r;
  FA_END
}

// ------------------------------------------------------------------ rope
// Checks that both directions share.
fa_rope_args rope_common(const at::Tensor *q, const at::Tensor *k, const at::Tensor *wq,
                         const at::Tensor *wk, const at::Tensor *cos_sin,
                         const at::Tensor *positions, double eps, bool interleaved) {
  const int64_t n = q->dim();
  if ((n != 3 && n != 4) || k->dim() != n || k->size(n - 1) != q->size(n - 1) ||
      k->sizes().slice(0, n - 2) != q->sizes().slice(0, n - 2))
    bad("%sq, k must be [T, H, D] and [T, H_kv, D], or [B, L, H, D] and [B, L, H_kv, D]");
  fa_rope_args r;
  std::memset(&r, 0, sizeof(r));
  r.dtype = dtype_of(q);
  r.B = n == 4 ? size32(q->size(0), "q") : 1;
  r.L = size32(q->size(n - 3), "q");
  r.H = size32(q->size(n - 2), "q");
  r.H_kv = size32(k->size(n - 2), "k");
  r.D = size32(q->size(n - 1), "q");
  const at::ScalarType type = q->scalar_type();
  if (wq) vec(wq, "q_weight", type, r.D);
  if (wk) vec(wk, "k_weight", type, r.D);
  if (cos_sin->dim() != 2 || cos_sin->scalar_type() != at::kFloat || !cos_sin->is_contiguous())
    bad("%scos_sin must be a contiguous float32 [max_pos, rot_dim]");
  const bool wide = positions->scalar_type() == at::kLong;
  if (positions->sizes() != q->sizes().slice(0, n - 2) ||
      !(wide || positions->scalar_type() == at::kInt))
    bad("%spositions must be int32 or int64 of q's token axes");
  r.q = rows_of(q, "q", q->sizes(), type);
  r.k = rows_of(k, "k", k->sizes(), type);
  r.q_weight = wq ? wq->data_ptr() : nullptr;
  r.k_weight = wk ? wk->data_ptr() : nullptr;
  r.cos_sin = static_cast<const float *>(cos_sin->data_ptr());
  r.max_pos = size32(cos_sin->size(0), "cos_sin");
  r.rot_dim = size32(cos_sin->size(1), "cos_sin");
  r.positions = positions->data_ptr();
  r.positions_64 = wide;
  r.positions_stride_b = n == 4 ? positions->stride(0) : 0;
  r.positions_stride_l = positions->stride(n - 3);
  r.interleaved = interleaved;
  r.eps = static_cast<float>(eps);
  return r;
}

// (q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, q_out, k_out, v, k_cache, v_cache, slots, stream)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t na) {
  FA_BEGIN
  count(na, 15);
  const at::Tensor *q = tensor(a[0], "q"), *k = tensor(a[1], "k"),
                   *wq = tensor(a[2], "q_weight", true), *wk = tensor(a[3], "k_weight", true),
                   *cs = tensor(a[4], "cos_sin"), *pos = tensor(a[5], "positions"),
                   *qo = tensor(a[8], "q_out", true), *ko = tensor(a[9], "k_out", true),
                   *v = tensor(a[10], "v", true), *kc = tensor(a[11], "k_cache", true),
                   *vc = tensor(a[12], "v_cache", true), *slots = tensor(a[13], "slots", true);
  fa_rope_args r = rope_common(q, k, wq, wk, cs, pos, real(a[6]), truth(a[7]));
  const at::ScalarType type = q->scalar_type();
  const bool cached = kc || vc;
  if (cached) {
    if (!kc || !vc || !v || !slots) bad("%sa cache needs k_cache, v_cache, v and slots");
    const Cache c = cache_of(kc, vc, r.H_kv, r.D, type);
    r.num_pages = c.pages;
    r.page_size = c.page_size;
    r.cache_stride_page = c.sp;
    r.cache_stride_token = c.st;
    r.cache_stride_head = c.sh;
    r.k_cache = kc->data_ptr();
    r.v_cache = vc->data_ptr();
    r.v = rows_of(v, "v", k->sizes(), type);
    if (slots->scalar_type() != at::kLong || slots->numel() != static_cast<int64_t>(r.B) * r.L ||
        !slots->is_contiguous())
      bad("%sslots must be contiguous int64, one per token");
    r.slots = static_cast<const long long *>(slots->data_ptr());
  }
  Device dev;
  const at::Tensor *all[12] = {q, k, wq, wk, cs, pos, qo, ko, v, kc, vc, slots};
  static const char *names[12] = {"q", "k", "q_weight", "k_weight", "cos_sin", "positions", "q_out",
                                  "k_out", "v", "k_cache", "v_cache", "slots"};
  for (int i = 0; i < 12; ++i) dev.on(all[i], names[i]);
  c10::cuda::CUDAGuard guard(dev.index);
  const Stream stream(a[14], dev.index);
  at::Tensor q_out, k_out;
  if (!qo) {
    q_out = empty(q->sizes(), q, type);
    qo = &q_out;
  }
  if (!ko && !cached) {
    k_out = empty(k->sizes(), q, type);
    ko = &k_out;
  }
  r.q_out = rows_of(qo, "q_out", q->sizes(), type);
  if (ko) r.k_out = rows_of(ko, "k_out", k->sizes(), type);
  call("fa_qk_norm_rope", [&] { return fa_qk_norm_rope(&r, stream.s); });
  PyObject *res = PyTuple_New(2);
  if (!res) return nullptr;
  if (q_out.defined()) {
    PyTuple_SET_ITEM(res, 0, THPVariable_Wrap(std::move(q_out)));
  } else {
    Py_INCREF(a[8]);
    PyTuple_SET_ITEM(res, 0, a[8]);
  }
  if (k_out.defined()) {
    PyTuple_SET_ITEM(res, 1, THPVariable_Wrap(std::move(k_out)));
  } else {
    Py_INCREF(a[9]);
    PyTuple_SET_ITEM(res, 1, a[9]);
  }
  return res;
  FA_END
}

// (q, k, q_weight, k_weight, cos_sin, positions, dq_out, dk_out, eps, interleaved, dq, dk, workspace, stream)
PyObject *qk_norm_rope_bwd(PyObject *, PyObject *const *a, Py_ssize_t na) {
  FA_BEGIN
  count(na, 14);
  const at::Tensor *q = tensor(a[0], "q"), *k = tensor(a[1], "k"),
                   *wq = tensor(a[2], "q_weight", true), *wk = tensor(a[3], "k_weight", true),
                   *cs = tensor(a[4], "cos_sin"), *pos = tensor(a[5], "positions"),
                   *dqo = tensor(a[6], "dq_out"), *dko = tensor(a[7], "dk_out"),
                   *dq = tensor(a[10], "dq", true), *dk = tensor(a[11], "dk", true),
                   *ws = tensor(a[12], "workspace", true);
  workspace(ws);
  fa_rope_args r = rope_common(q, k, wq, wk, cs, pos, real(a[8]), truth(a[9]));
  const at::ScalarType type = q->scalar_type();
  r.q_out = rows_of(dqo, "dq_out", q->sizes(), type);
  r.k_out = rows_of(dko, "dk_out", k->sizes(), type);
  Device dev;
  const at::Tensor *all[11] = {q, k, wq, wk, cs, pos, dqo, dko, dq, dk, ws};
  static const char *names[11] = {"q", "k", "q_weight", "k_weight", "cos_sin", "positions", "dq_out",
                                  "dk_out", "dq", "dk", "workspace"};
  for (int i = 0; i < 11; ++i) dev.on(all[i], names[i]);
  c10::cuda::CUDAGuard guard(dev.index);
  const Stream stream(a[13], dev.index);
  at::Tensor o[4];   // dq, dk, dq_weight, dk_weight
  if (dq) o[0] = *dq; else o[0] = empty(q->sizes(), q, type);
  if (dk) o[1] = *dk; else o[1] = empty(k->sizes(), q, type);
  const fa_rows rq = rows_of(&o[0], "dq", q->sizes(), type), rk = rows_of(&o[1], "dk", k->sizes(), type);
  // the weight gradients (one allocation) and, unless given, the workspace
  if (wq || wk) {
    const at::Tensor both = empty({2ll * r.D}, q, at::kFloat);
    if (wq) o[2] = part(both, at::kFloat, 0, r.D);
    if (wk) o[3] = part(both, at::kFloat, r.D, r.D);
  }
  at::Tensor own;
  if (!ws && (wq || wk)) {
    own = empty({static_cast<int64_t>(fa_qk_norm_rope_bwd_workspace_bytes(r.D))}, q, at::kByte);
    ws = &own;
  }
  call("fa_qk_norm_rope_bwd", [&] {
    return fa_qk_norm_rope_bwd(&r, rq, rk, wq ? static_cast<float *>(o[2].data_ptr()) : nullptr,
                               wk ? static_cast<float *>(o[3].data_ptr()) : nullptr,
                               ws ? ws->data_ptr() : nullptr,
                               ws ? static_cast<size_t>(ws->numel()) * ws->element_size() : 0,
                               stream.s);
  });
  PyObject *res = PyTuple_New(4);
  for (int i = 0; res && i < 4; ++i) {
    if (o[i].defined()) {
      PyTuple_SET_ITEM(res, i, THPVariable_Wrap(std::move(o[i])));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(res, i, Py_None);
    }
  }
  return res;
  FA_END
}

// ------------------------------------------------------------------ flash_fwd_paged
// (q, k_cache, v_cache, block_table, cu_q, kv_lens, scale | None, causal, window_left, window_right,
//  return_lse, out, lse, workspace, stream)
PyObject *flash_fwd_paged(PyObject *, PyObject *const *a, Py_ssize_t na) {
  FA_BEGIN
  count(na, 15);
  const at::Tensor *q = tensor(a[0], "q"), *k = tensor(a[1], "k_cache"), *v = tensor(a[2], "v_cache"),
                   *table = tensor(a[3], "block_table"), *cu = tensor(a[4], "cu_q"),
                   *kv = tensor(a[5], "kv_lens"), *out = tensor(a[11], "out", true),
                   *lse = tensor(a[12], "lse", true), *ws = tensor(a[13], "workspace", true);
  workspace(ws);
  if (q->dim() != 3 || q->stride(2) != 1) bad("%sq must be [total_q, H, D], contiguous along D");
  const int T = size32(q->size(0), "q"), H = size32(q->size(1), "q"), D = size32(q->size(2), "q");
  const int dtype = dtype_of(q);
  const at::ScalarType type = q->scalar_type();
  if (k->dim() != 4 || kv->dim() != 1)
    bad("%sk_cache, v_cache must be [pages, page_size, H_kv, D], kv_lens a vector");
  const int H_kv = size32(k->size(2), "k_cache"), B = size32(kv->size(0), "kv_lens");
  const Cache c = cache_of(k, v, H_kv, D, type);
  vec(kv, "kv_lens", at::kInt, B);
  vec(cu, "cu_q", at::kInt, B + 1ll);
  const Table tb = table_of(table, B);
  const float scale = a[6] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)))
                                      : static_cast<float>(real(a[6]));
  const int causal = truth(a[7]), wl = int32(a[8], "window_left"), wr = int32(a[9], "window_right");
  const bool want_lse = truth(a[10]);
  Device dev;
  const at::Tensor *all[9] = {q, k, v, table, cu, kv, out, lse, ws};
  static const char *names[9] = {"q", "k_cache", "v_cache", "block_table", "cu_q", "kv_lens", "out",
                                 "lse", "workspace"};
  for (int i = 0; i < 9; ++i) dev.on(all[i], names[i]);
  c10::cuda::CUDAGuard guard(dev.index);
  const Stream stream(a[14], dev.index);
  at::Tensor o, l, own;
  if (!out) {
    o = empty(q->sizes(), q, type);
    out = &o;
  } else if (out->sizes() != q->sizes() || out->scalar_type() != type || out->stride(2) != 1) {
    bad("%sout must be like q, contiguous along D");
  }
  if (!want_lse) {
    lse = nullptr;
  } else if (!lse) {
    l = empty({T, H}, q, at::kFloat);
    lse = &l;
  } else if (lse->dim() != 2 || lse->size(0) != T || lse->size(1) != H ||
             lse->scalar_type() != at::kFloat || !lse->is_contiguous()) {
    bad("%slse must be a contiguous float32 [total_q, H]");
  }
  if (!ws) {
    own = empty({static_cast<int64_t>(fa_paged_workspace_bytes(D)) + 1}, q, at::kByte);
    ws = &own;
  }
  call("fa_fwd_paged", [&] {
    return fa_fwd_paged(q->data_ptr(), q->stride(0), q->stride(1), k->data_ptr(), v->data_ptr(), c.sp,
                        c.st, c.sh, static_cast<int *>(table->data_ptr()), tb.stride,
                        static_cast<int *>(cu->data_ptr()), static_cast<int *>(kv->data_ptr()),
                        out->data_ptr(), out->stride(0), out->stride(1),
                        lse ? static_cast<float *>(lse->data_ptr()) : nullptr, T, B, H, H_kv, D,
                        c.pages, c.page_size, tb.columns, scale, causal, wl, wr, dtype,
                        ws->data_ptr(), static_cast<size_t>(ws->numel()) * ws->element_size(),
                        stream.s);
  });
  PyObject *res = PyTuple_New(2);
  if (!res) return nullptr;
  if (o.defined()) {
    PyTuple_SET_ITEM(res, 0, THPVariable_Wrap(std::move(o)));
  } else {
    Py_INCREF(a[11]);
    PyTuple_SET_ITEM(res, 0, a[11]);
  }
  if (l.defined()) {
    PyTuple_SET_ITEM(res, 1, THPVariable_Wrap(std::move(l)));
  } else {
    PyObject *given = lse ? a[12] : Py_None;
    Py_INCREF(given);
    PyTuple_SET_ITEM(res, 1, given);
  }
  return res;
  FA_END
}

PyObject *set_error(PyObject *, PyObject *type) {
  Py_XINCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"paged_plan", fast(paged_plan), METH_FASTCALL, nullptr},
    {"qk_norm_rope", fast(qk_norm_rope), METH_FASTCALL, nullptr},
    {"qk_norm_rope_bwd", fast(qk_norm_rope_bwd), METH_FASTCALL, nullptr},
    {"flash_fwd_paged", fast(flash_fwd_paged), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch(void) { return PyModule_Create(&module); }
