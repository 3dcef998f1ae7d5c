// The serving calls' short way from Python, for the usual arguments: tensors of
// the right type and layout on the current device, no stream given.  A step's
// single-token calls take a few microseconds on the GPU, and reading a dozen
// tensors' shapes and addresses through Python and ctypes, with caches that
// the last launch has emptied, takes longer than that: one token of SWA 16.7 us
// a call against 4.6 to 6.2 here (4.1 on the GPU), a plan of 64 tokens 28 against
// 5.9, an append of 128 tokens 19 against 6.0.  Whatever is not as expected returns
// None, and the caller goes the long way, which says what is wrong.  The
// functions of libsa.so are handed over by address (bind).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "libsa.h"

namespace {

decltype(&swa_paged_forward) g_swa;
decltype(&sa_paged_forward) g_sa;
decltype(&sa_swa_gated_paged_forward) g_gated;
decltype(&sa_paged_workspace_size) g_workspace;
decltype(&sa_paged_plan) g_plan;
decltype(&sa_paged_append) g_append;

// A tensor argument: exactly a torch.Tensor, dense, on device `dev` (-1: the
// first one seen sets it).
struct Args {
  int dev = -1;
  bool ok = true;
  const at::Tensor* tensor(PyObject* o, at::ScalarType type, int64_t dim) {
    if (!ok || !THPVariable_CheckExact(o)) return no();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || t.dim() != dim || t.layout() != at::kStrided || !t.is_cuda()) return no();
    const int d = t.get_device();
    if (dev < 0) dev = d;
    if (d != dev) return no();
    return &t;
  }
  const at::Tensor* dense(PyObject* o, at::ScalarType type, int64_t dim) {
    const at::Tensor* t = tensor(o, type, dim);
    return t == nullptr || !t->is_contiguous() ? no() : t;
  }
  // [T, H, d] with contiguous rows [H, d]; the stride between tokens
  const at::Tensor* tokens(PyObject* o, int64_t* stride) {
    const at::Tensor* t = tensor(o, at::kBFloat16, 3);
    if (t == nullptr) return no();
    const int64_t n = t->size(0), h = t->size(1), d = t->size(2);
    *stride = h * d;
    if (t->is_contiguous()) return t;
    if ((t->stride(2) != 1 && d > 1) || (t->stride(1) != d && h > 1) || (t->stride(0) < h * d && n > 1)) return no();
    if (n > 1) *stride = t->stride(0);
    return t;
  }
  // both caches [pages, page, Hkv, d], pages the same stride apart
  bool caches(PyObject* ko, PyObject* vo, const at::Tensor** k, const at::Tensor** v, int64_t* stride) {
    *k = tensor(ko, at::kBFloat16, 4);
    *v = tensor(vo, at::kBFloat16, 4);
    if (!ok || (*k)->sizes() != (*v)->sizes() || (*k)->numel() == 0) return no() != nullptr;
    const int64_t h = (*k)->size(2), d = (*k)->size(3), size = (*k)->size(1) * h * d;
    *stride = size;
    if ((*k)->is_contiguous() && (*v)->is_contiguous()) return true;
    for (const at::Tensor* t : {*k, *v}) {
      if (t->stride(3) != 1 || t->stride(2) != d || t->stride(1) != h * d || t->stride(0) < size) return no() != nullptr;
    }
    if ((*k)->stride(0) != (*v)->stride(0)) return no() != nullptr;
    *stride = (*k)->stride(0);
    return true;
  }
  int32_t* err(PyObject* o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o) || THPVariable_Unpack(o).numel() < 1) return (no(), nullptr);
    const at::Tensor* t = tensor(o, at::kInt, THPVariable_Unpack(o).dim());
    return t ? static_cast<int32_t*>(t->data_ptr()) : nullptr;
  }
  int32_t integer(PyObject* o) {
    if (!PyLong_CheckExact(o)) return (no(), 0);
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &over);
    if (over != 0 || x < INT32_MIN || x > INT32_MAX) return (no(), 0);
    return int32_t(x);
  }
  double real(PyObject* o) {
    if (!PyFloat_CheckExact(o)) return double(integer(o));
    return PyFloat_AS_DOUBLE(o);
  }
  bool here() {  // everything is as expected, and its device the current one
    return ok && dev >= 0 && c10::cuda::current_device() == dev;
  }
  const at::Tensor* no() {
    ok = false;
    return nullptr;
  }
};

int32_t* ints(const at::Tensor* t) { return static_cast<int32_t*>(t->data_ptr()); }
cudaStream_t stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream(); }
bool fits(int64_t x) { return x <= INT32_MAX; }

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[6] = {};
  for (Py_ssize_t i = 0; i < n && i < 6; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  g_swa = reinterpret_cast<decltype(g_swa)>(p[0]);
  g_sa = reinterpret_cast<decltype(g_sa)>(p[1]);
  g_gated = reinterpret_cast<decltype(g_gated)>(p[2]);
  g_workspace = reinterpret_cast<decltype(g_workspace)>(p[3]);
  g_plan = reinterpret_cast<decltype(g_plan)>(p[4]);
  g_append = reinterpret_cast<decltype(g_append)>(p[5]);
  Py_RETURN_NONE;
}

// (path, q, k_cache, v_cache, block_table, q_start, seq_lens, window, window_swa,
// max_new, softmax_scale, out, kernel, err, perm, inv_perm, gate_sa, gate_swa)
// -> out, a status other than 0, or None.
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 18 || g_swa == nullptr) Py_RETURN_NONE;
  Args x;
  sa_paged_params_t p = {};
  const at::Tensor *k, *v, *perm = nullptr, *inv = nullptr, *gs = nullptr, *gw = nullptr, *given = nullptr;
  const int path = x.integer(a[0]);
  const at::Tensor* q = x.tokens(a[1], &p.q_stride);
  if (!x.caches(a[2], a[3], &k, &v, &p.page_stride)) Py_RETURN_NONE;
  const at::Tensor* table = x.dense(a[4], at::kInt, 2);
  const at::Tensor* q_start = x.dense(a[5], at::kInt, 1);
  const at::Tensor* lens = x.dense(a[6], at::kInt, 1);
  p.window = x.integer(a[7]);
  p.window_swa = x.integer(a[8]);
  p.max_new = x.integer(a[9]);
  p.softmax_scale = float(x.real(a[10]));
  if (a[11] != Py_None) given = x.dense(a[11], at::kBFloat16, 3);
  p.kernel = x.integer(a[12]);
  p.err = x.err(a[13]);
  if (path != 0) {
    perm = x.dense(a[14], at::kInt, 2);
    inv = x.dense(a[15], at::kInt, 2);
  }
  if (path == 2) {
    gs = x.dense(a[16], at::kFloat, 2);
    gw = x.dense(a[17], at::kFloat, 2);
  }
  if (!x.here()) Py_RETURN_NONE;
  const int64_t T = q->size(0), Hq = q->size(1), d = q->size(2), B = lens->size(0);
  if (k->size(3) != d || table->size(0) != B || q_start->size(0) != B + 1) Py_RETURN_NONE;
  if (perm && (inv->sizes() != perm->sizes() || (perm->size(0) != B && perm->size(0) != 1))) Py_RETURN_NONE;
  if (gs && (gs->size(0) != T || gs->size(1) != Hq || gw->sizes() != gs->sizes())) Py_RETURN_NONE;
  if (given && given->sizes() != q->sizes()) Py_RETURN_NONE;
  if (!fits(T) || !fits(Hq) || !fits(d) || !fits(B) || !fits(k->size(0)) || !fits(k->size(1)) || !fits(k->size(2)) ||
      !fits(table->size(1)) || (perm && !fits(perm->size(1))))
    Py_RETURN_NONE;
  p.batch = int32_t(B);
  p.tokens = int32_t(T);
  p.num_q_heads = int32_t(Hq);
  p.num_kv_heads = int32_t(k->size(2));
  p.head_dim = int32_t(d);
  p.page_size = int32_t(k->size(1));
  p.num_pages = int32_t(k->size(0));
  p.max_pages = int32_t(table->size(1));
  if (perm) {
    p.perm_rows = int32_t(perm->size(0));
    p.perm_len = int32_t(perm->size(1));
  }
  p.block_table = ints(table);
  p.q_start = ints(q_start);
  p.seq_lens = ints(lens);
  at::Tensor made, work;
  if (!given) {
    made = at::empty(q->sizes(), at::TensorOptions().dtype(at::kBFloat16).device(q->device()));
    given = &made;
  }
  const size_t bytes = g_workspace(&p, path);
  if (bytes > 0) work = at::empty({int64_t(bytes)}, at::TensorOptions().dtype(at::kByte).device(q->device()));
  void* const ws = bytes > 0 ? work.data_ptr() : nullptr;
  const cudaStream_t s = stream_of(x.dev);
  void *const qp = q->data_ptr(), *const kp = k->data_ptr(), *const vp = v->data_ptr(), *const op = given->data_ptr();
  const sa_status_t st =
      path == 0   ? g_swa(&p, qp, kp, vp, op, ws, bytes, s)
      : path == 1 ? g_sa(&p, qp, kp, vp, ints(perm), ints(inv), op, ws, bytes, s)
                  : g_gated(&p, qp, kp, vp, ints(perm), ints(inv), static_cast<const float*>(gs->data_ptr()),
                            static_cast<const float*>(gw->data_ptr()), op, ws, bytes, s);
  if (st != SA_OK) return PyLong_FromLong(st);
  if (made.defined()) return THPVariable_Wrap(std::move(made));
  return Py_NewRef(a[11]);
  END_HANDLE_TH_ERRORS
}

// (new_lens, cached_lens, block_table, free_pages, num_free, page_size, num_pages,
// max_tokens, err) -> (q_start, seq_lens, slots, positions, counts), a status, or None.
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9 || g_plan == nullptr) Py_RETURN_NONE;
  Args x;
  const at::Tensor* now = x.dense(a[0], at::kInt, 1);
  const at::Tensor* cached = x.dense(a[1], at::kInt, 1);
  const at::Tensor* table = x.dense(a[2], at::kInt, 2);
  const at::Tensor* free = x.dense(a[3], at::kInt, 1);
  const at::Tensor* num = x.dense(a[4], at::kInt, 1);
  const int page = x.integer(a[5]), pages = x.integer(a[6]), most = x.integer(a[7]);
  int32_t* err = x.err(a[8]);
  if (!x.here()) Py_RETURN_NONE;
  const int64_t B = now->size(0);
  if (cached->size(0) != B || table->size(0) != B || num->size(0) != 1 || most < 0 || !fits(B) ||
      !fits(table->size(1)) || !fits(free->size(0)))
    Py_RETURN_NONE;
  // the five outputs are pieces of one allocation
  const int64_t sizes[5] = {B + 1, B, most, most, 3};
  const at::Tensor all =
      at::empty({2 * B + 1 + 2 * int64_t(most) + 3}, at::TensorOptions().dtype(at::kInt).device(now->device()));
  int32_t* out[5];
  int64_t at0[5], at_ = 0;
  for (int i = 0; i < 5; ++i) {
    at0[i] = at_;
    out[i] = ints(&all) + at_;
    at_ += sizes[i];
  }
  const sa_status_t st = g_plan(ints(now), ints(cached), int32_t(B), ints(table), int32_t(table->size(1)), ints(free),
                                int32_t(free->size(0)), ints(num), page, pages, most, out[0], out[1], out[2], out[3],
                                out[4], err, stream_of(x.dev));
  if (st != SA_OK) return PyLong_FromLong(st);
  PyObject* tuple = PyTuple_New(5);
  if (tuple == nullptr) return nullptr;
  for (int i = 0; i < 5; ++i) {
    at::Tensor t =
        at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(at0[i]);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(&sizes[i], 1));
    PyTuple_SET_ITEM(tuple, i, THPVariable_Wrap(std::move(t)));
  }
  return tuple;
  END_HANDLE_TH_ERRORS
}

// (k, v, k_cache, v_cache, slots, positions, rope_base, q, q_out, err) -> q_out,
// True where there is none, a status, or None.
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10 || g_append == nullptr) Py_RETURN_NONE;
  Args x;
  sa_paged_append_params_t p = {};
  const at::Tensor *kc, *vc, *pos = nullptr, *q = nullptr, *given = nullptr;
  const at::Tensor* k = x.tokens(a[0], &p.k_stride);
  const at::Tensor* v = x.tokens(a[1], &p.v_stride);
  if (!x.caches(a[2], a[3], &kc, &vc, &p.page_stride)) Py_RETURN_NONE;
  const at::Tensor* slots = x.dense(a[4], at::kInt, 1);
  if (a[5] != Py_None) pos = x.dense(a[5], at::kInt, 1);
  p.rope_base = x.real(a[6]);
  if (a[7] != Py_None) q = x.tokens(a[7], &p.q_stride);
  if (a[8] != Py_None) given = x.dense(a[8], at::kBFloat16, 3);
  p.err = x.err(a[9]);
  if (!x.here()) Py_RETURN_NONE;
  const int64_t T = k->size(0), h = k->size(1), d = k->size(2);
  const bool rope = p.rope_base != 0.0;
  if (v->sizes() != k->sizes() || kc->size(2) != h || kc->size(3) != d || slots->size(0) != T ||
      (pos && pos->size(0) != T) || (rope && !pos) || (q && !rope) || (given && !q))
    Py_RETURN_NONE;
  if (q && (q->size(0) != T || q->size(2) != d || (given && given->sizes() != q->sizes()))) Py_RETURN_NONE;
  if (!fits(T) || !fits(h) || !fits(d) || (q && !fits(q->size(1))) || !fits(kc->size(0)) || !fits(kc->size(1)))
    Py_RETURN_NONE;
  p.tokens = int32_t(T);
  p.num_kv_heads = int32_t(h);
  p.num_q_heads = q ? int32_t(q->size(1)) : 0;
  p.head_dim = int32_t(d);
  p.page_size = int32_t(kc->size(1));
  p.num_pages = int32_t(kc->size(0));
  at::Tensor made;
  if (q && !given) {
    made = at::empty(q->sizes(), at::TensorOptions().dtype(at::kBFloat16).device(q->device()));
    given = &made;
  }
  const sa_status_t st = g_append(&p, k->data_ptr(), v->data_ptr(), q ? q->data_ptr() : nullptr, ints(slots),
                                  rope ? ints(pos) : nullptr, kc->data_ptr(), vc->data_ptr(),
                                  q ? given->data_ptr() : nullptr, stream_of(x.dev));
  if (st != SA_OK) return PyLong_FromLong(st);
  if (!q) Py_RETURN_TRUE;
  if (made.defined()) return THPVariable_Wrap(std::move(made));
  return Py_NewRef(a[8]);
  END_HANDLE_TH_ERRORS
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(forward)), METH_FASTCALL, nullptr},
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged_call", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_call() { return PyModule_Create(&g_module); }
