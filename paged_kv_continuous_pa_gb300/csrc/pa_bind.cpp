// pa_bind.cpp -- the Python binding's short way for calls whose arguments are as they
// should be: tensors are looked at and the C ABI is called in one step.  In a serving loop these
// calls stand beside kernels of a few microseconds; the same looks through Python attributes
// and ctypes took 9 of a call's 13 us (12 tensors), here they take about one.
//
// Each function returns the call's status, or None, with nothing done, where an argument is not of
// the plain kind (another type, shape, layout or device, a stream of the caller's): the
// binding then goes the long way, which raises the errors or makes the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>

#include "../../include/pa.h"

namespace {

decltype(&pa_append_kv) f_append;
decltype(&pa_attention) f_attention;
decltype(&pa_tables_grow) f_tables_grow;
decltype(&pa_rope_append) f_rope_append;
decltype(&pa_prompt_attention) f_prompt;
decltype(&pa_read_kv) f_read;

constexpr auto I32 = at::kInt;

// The arguments of a call; `ok` turns false with the first that is not of the plain kind.
struct Args {
  PyObject* const* a;
  bool ok;
  int device = -1;

  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : a(args), ok(n == want) {}

  bool none(int i) const { return a[i] == Py_None; }
  const at::Tensor* tensor(int i) {
    if (!ok || !THPVariable_CheckExact(a[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided) return fail();
    const int d = t.get_device();
    if (device < 0) device = d;
    if (d != device) return fail();
    for (const int64_t s : t.sizes())
      if (s > INT_MAX) return fail();
    return &t;
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  // a contiguous tensor of `dims` dimensions; its address
  void* dense(int i, c10::optional<at::ScalarType> type, int dims, const at::Tensor** out = nullptr) {
    const at::Tensor* t = tensor(i);
    if (t == nullptr || (type && t->scalar_type() != *type) || (dims > 0 && t->dim() != dims) || !t->is_contiguous()) {
      fail();
      return nullptr;
    }
    if (out != nullptr) *out = t;
    return t->data_ptr();
  }
  // int32 [n]
  int32_t* list(int i, int64_t n) {
    const at::Tensor* t = nullptr;
    void* p = dense(i, I32, 1, &t);
    if (t != nullptr && t->size(0) != n) fail();
    return static_cast<int32_t*>(p);
  }
  int32_t* optional_list(int i) { return none(i) ? nullptr : static_cast<int32_t*>(dense(i, I32, 1)); }
  bool shape(const at::Tensor* t, std::initializer_list<int64_t> want) {
    if (t == nullptr || t->sizes() != c10::IntArrayRef(want)) ok = false;
    return ok;
  }
  // rows [n, heads, D] with contiguous heads; the elements from row to row
  void* rows(int i, const at::Tensor** out, int64_t* stride) {
    const at::Tensor* t = tensor(i);
    if (t == nullptr || t->dim() != 3) {
      fail();
      return nullptr;
    }
    const int64_t n = t->size(0), heads = t->size(1), d = t->size(2);
    if ((d > 1 && t->stride(2) != 1) || (heads > 1 && t->stride(1) != d)) {
      fail();
      return nullptr;
    }
    *stride = n > 1 ? t->stride(0) : heads * d;
    *out = t;
    return t->data_ptr();
  }
  long long number(int i) {
    const long long v = PyLong_Check(a[i]) ? PyLong_AsLongLong(a[i]) : (ok = false, 0);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  int32_t number32(int i) {
    const long long v = number(i);
    if (v < INT_MIN || v > INT_MAX) ok = false;
    return static_cast<int32_t>(v);
  }
  // the address of a live handle
  void* address(int i) {
    const long long v = number(i);
    if (v == 0) ok = false;
    return reinterpret_cast<void*>(static_cast<uintptr_t>(v));
  }
  float real(int i) {
    const double v = PyFloat_Check(a[i]) ? PyFloat_AS_DOUBLE(a[i]) : (ok = false, 0.0);
    return static_cast<float>(v);
  }
  // f32 or bf16
  pa_dtype dtype(const at::Tensor* t) {
    if (t != nullptr && t->scalar_type() == at::kBFloat16) return PA_BF16;
    if (t == nullptr || t->scalar_type() != at::kFloat) ok = false;
    return PA_F32;
  }
  // the device's current stream, where that is the current device
  void* stream() {
    if (!ok || device != c10::cuda::current_device()) {
      ok = false;
      return nullptr;
    }
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  }
};

// The call itself, without the interpreter's lock: a launch may wait for a place in the stream's
// queue, and what the stream waits for may need the lock.
template <class F, class... A>
PyObject* call(F f, A... args) {
  PyThreadState* state = PyEval_SaveThread();
  const pa_status st = f(args...);
  PyEval_RestoreThread(state);
  return PyLong_FromLong(static_cast<long>(st));
}

#define PA_SHORT_WAY_CHECK(x) \
  if (!(x).ok) Py_RETURN_NONE

// pool address, kv heads, head_dim, pool tensor, k_new, v_new, seq_ids, positions, block_tables, status
PyObject* append_kv(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  Args x(args, n_args, 10);
  PA_SHORT_WAY_CHECK(x);
  const at::Tensor *k, *v, *tables;
  const void* pool = x.address(0);
  const int64_t heads = x.number(1), d = x.number(2);
  x.tensor(3);
  const void* kp = x.dense(4, c10::nullopt, 3, &k);
  const void* vp = x.dense(5, c10::nullopt, 3, &v);
  const int32_t* tp = static_cast<int32_t*>(x.dense(8, I32, 2, &tables));
  PA_SHORT_WAY_CHECK(x);
  const int64_t n = k->size(0);
  const int32_t *ids = x.list(6, n), *positions = x.list(7, n);
  int32_t* status = x.optional_list(9);
  const pa_dtype type = x.dtype(k);
  if (!x.shape(k, {n, heads, d}) || !x.shape(v, {n, heads, d}) || v->scalar_type() != k->scalar_type()) Py_RETURN_NONE;
  void* stream = x.stream();
  PA_SHORT_WAY_CHECK(x);
  return call(f_append, static_cast<const pa_pool*>(pool), static_cast<int32_t>(n), kp, vp, type, ids, positions, tp,
                         static_cast<int32_t>(tables->size(0)), static_cast<int32_t>(tables->size(1)), status, stream);
}

// pool address, head_dim, pool tensor, q, seq_ids, positions, block_tables, out, softmax_scale, workspace, status (no chunks)
PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  Args x(args, n_args, 11);
  PA_SHORT_WAY_CHECK(x);
  const at::Tensor *q, *tables, *out, *ws = nullptr;
  const void* pool = x.address(0);
  const int64_t d = x.number(1);
  x.tensor(2);
  const void* qp = x.dense(3, c10::nullopt, 3, &q);
  const int32_t* tp = static_cast<int32_t*>(x.dense(6, I32, 2, &tables));
  void* op = x.dense(7, c10::nullopt, 3, &out);
  void* wp = x.none(9) ? nullptr : x.dense(9, c10::nullopt, 0, &ws);
  PA_SHORT_WAY_CHECK(x);
  const int64_t n = q->size(0);
  const int32_t *ids = x.list(4, n), *positions = x.list(5, n);
  int32_t* status = x.optional_list(10);
  const float scale = x.real(8);
  const pa_dtype type = x.dtype(q);
  if (!x.shape(q, {n, q->size(1), d}) || !x.shape(out, {n, q->size(1), d}) || out->scalar_type() != q->scalar_type()) Py_RETURN_NONE;
  void* stream = x.stream();
  PA_SHORT_WAY_CHECK(x);
  return call(f_attention, static_cast<const pa_pool*>(pool), static_cast<int32_t>(n), qp, type, static_cast<int32_t>(q->size(1)),
                            ids, positions, tp, static_cast<int32_t>(tables->size(0)), static_cast<int32_t>(tables->size(1)),
                            nullptr, 0, scale, op, wp, ws == nullptr ? 0 : ws->nbytes(), status, stream);
}

// seq_ids, lengths, new_tokens, free_pages, free_count, free_left, page_size, block_tables, row_starts, page_starts, row_seqs,
// row_positions, row_slots, status
PyObject* tables_grow(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  Args x(args, n_args, 14);
  PA_SHORT_WAY_CHECK(x);
  const at::Tensor *ids, *free_pages, *tables, *row_seqs, *slots = nullptr;
  const int32_t* ip = static_cast<int32_t*>(x.dense(0, I32, 1, &ids));
  const int32_t* fp = static_cast<int32_t*>(x.dense(3, I32, 1, &free_pages));
  int32_t* tp = static_cast<int32_t*>(x.dense(7, I32, 2, &tables));
  int32_t* rp = static_cast<int32_t*>(x.dense(10, I32, 1, &row_seqs));
  int64_t* sp = x.none(12) ? nullptr : static_cast<int64_t*>(x.dense(12, at::kLong, 1, &slots));
  PA_SHORT_WAY_CHECK(x);
  const int64_t n = ids->size(0), rows = row_seqs->size(0);
  const int32_t *lengths = x.list(1, n), *more = x.list(2, n), *count = x.list(4, 1);
  int32_t *left = x.list(5, 1), *row_starts = x.list(8, n + 1), *page_starts = x.list(9, n + 1), *positions = x.list(11, rows);
  int32_t* status = x.optional_list(13);
  const int32_t page = x.number32(6);
  if (slots != nullptr && slots->size(0) != rows) Py_RETURN_NONE;
  void* stream = x.stream();
  PA_SHORT_WAY_CHECK(x);
  return call(f_tables_grow, static_cast<int32_t>(n), ip, lengths, more, fp, count, left, static_cast<int32_t>(free_pages->size(0)), page,
                              tp, static_cast<int32_t>(tables->size(0)), static_cast<int32_t>(tables->size(1)), row_starts,
                              page_starts, static_cast<int32_t>(rows), rp, positions, sp, status, stream);
}

// pool address, kv heads, head_dim, pool tensor, rope address or None, q, k, v, seq_ids, positions, block_tables, q_out, status
PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  Args x(args, n_args, 13);
  PA_SHORT_WAY_CHECK(x);
  const at::Tensor *q = nullptr, *k = nullptr, *v = nullptr, *out = nullptr, *tables;
  const void *pool = x.address(0), *rope = x.none(4) ? nullptr : x.address(4);
  const int64_t heads = x.number(1), d = x.number(2);
  x.tensor(3);
  int64_t q_stride = 0, k_stride = 0, v_stride = 0;
  const bool queries = !x.none(5);
  if (queries == x.none(11)) Py_RETURN_NONE;
  const void* qp = queries ? x.rows(5, &q, &q_stride) : nullptr;
  const void* kp = x.rows(6, &k, &k_stride);
  const void* vp = x.rows(7, &v, &v_stride);
  const int32_t* tp = static_cast<int32_t*>(x.dense(10, I32, 2, &tables));
  void* op = queries ? x.dense(11, c10::nullopt, 3, &out) : nullptr;
  PA_SHORT_WAY_CHECK(x);
  const int64_t n = k->size(0);
  const int32_t *ids = x.list(8, n), *positions = x.list(9, n);
  int32_t* status = x.optional_list(12);
  const pa_dtype type = x.dtype(k);
  if (!x.shape(k, {n, heads, d}) || !x.shape(v, {n, heads, d}) || v->scalar_type() != k->scalar_type()) Py_RETURN_NONE;
  if (queries && (!x.shape(q, {n, q->size(1), d}) || !x.shape(out, {n, q->size(1), d}) || q->scalar_type() != k->scalar_type() ||
                  out->scalar_type() != k->scalar_type()))
    Py_RETURN_NONE;
  void* stream = x.stream();
  PA_SHORT_WAY_CHECK(x);
  return call(f_rope_append, static_cast<const pa_pool*>(pool), static_cast<const pa_rope*>(rope), static_cast<int32_t>(n), qp,
                              q_stride, queries ? static_cast<int32_t>(q->size(1)) : 0, op, kp, k_stride, vp, v_stride, type, ids,
                              positions, tp, static_cast<int32_t>(tables->size(0)), static_cast<int32_t>(tables->size(1)), status,
                              stream);
}

// q, k, v, row_starts, out, lse, softmax_scale, workspace, status
PyObject* prompt_attention(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  Args x(args, n_args, 9);
  PA_SHORT_WAY_CHECK(x);
  const at::Tensor *q = nullptr, *k = nullptr, *v = nullptr, *starts, *out, *lse = nullptr, *ws = nullptr;
  int64_t q_stride = 0, k_stride = 0, v_stride = 0;
  const void* qp = x.rows(0, &q, &q_stride);
  const void* kp = x.rows(1, &k, &k_stride);
  const void* vp = x.rows(2, &v, &v_stride);
  const int32_t* sp = static_cast<int32_t*>(x.dense(3, I32, 1, &starts));
  void* op = x.dense(4, c10::nullopt, 3, &out);
  float* lp = x.none(5) ? nullptr : static_cast<float*>(x.dense(5, at::kFloat, 2, &lse));
  void* wp = x.none(7) ? nullptr : x.dense(7, c10::nullopt, 0, &ws);
  int32_t* status = x.optional_list(8);
  const float scale = x.real(6);
  PA_SHORT_WAY_CHECK(x);
  const int64_t n = q->size(0), hq = q->size(1), d = q->size(2), hkv = k->size(1);
  const pa_dtype type = x.dtype(q);
  if (!x.shape(k, {n, hkv, d}) || !x.shape(v, {n, hkv, d}) || !x.shape(out, {n, hq, d}) || (lse != nullptr && !x.shape(lse, {n, hq})) ||
      k->scalar_type() != q->scalar_type() || v->scalar_type() != q->scalar_type() || out->scalar_type() != q->scalar_type() ||
      starts->size(0) < 1)
    Py_RETURN_NONE;
  void* stream = x.stream();
  PA_SHORT_WAY_CHECK(x);
  return call(f_prompt, static_cast<int32_t>(n), static_cast<int32_t>(starts->size(0) - 1), qp, q_stride, kp, k_stride, vp, v_stride,
                         type, static_cast<int32_t>(hq), static_cast<int32_t>(hkv), static_cast<int32_t>(d), sp, scale, op, lp, wp,
                         ws == nullptr ? 0 : ws->nbytes(), status, stream);
}

// pool address, kv heads, head_dim, pool tensor, seq_ids, positions, block_tables, k_out, v_out, status
PyObject* read_kv(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  Args x(args, n_args, 10);
  PA_SHORT_WAY_CHECK(x);
  const at::Tensor *ids, *tables, *k = nullptr, *v = nullptr;
  const void* pool = x.address(0);
  const int64_t heads = x.number(1), d = x.number(2);
  x.tensor(3);
  const int32_t* ip = static_cast<int32_t*>(x.dense(4, I32, 1, &ids));
  const int32_t* tp = static_cast<int32_t*>(x.dense(6, I32, 2, &tables));
  void* kp = x.none(7) ? nullptr : x.dense(7, c10::nullopt, 3, &k);
  void* vp = x.none(8) ? nullptr : x.dense(8, c10::nullopt, 3, &v);
  PA_SHORT_WAY_CHECK(x);
  if (k == nullptr && v == nullptr) Py_RETURN_NONE;
  const int64_t n = ids->size(0);
  const int32_t* positions = x.list(5, n);
  int32_t* status = x.optional_list(9);
  const at::Tensor* out = k != nullptr ? k : v;
  const pa_dtype type = x.dtype(out);
  if ((k != nullptr && !x.shape(k, {n, heads, d})) ||
      (v != nullptr && (!x.shape(v, {n, heads, d}) || v->scalar_type() != out->scalar_type())))
    Py_RETURN_NONE;
  void* stream = x.stream();
  PA_SHORT_WAY_CHECK(x);
  return call(f_read, static_cast<const pa_pool*>(pool), static_cast<int32_t>(n), ip, positions, tp,
                       static_cast<int32_t>(tables->size(0)), static_cast<int32_t>(tables->size(1)), kp, vp, type, status, stream);
}

// Addresses of the library's functions, in the order below.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  Args x(args, n_args, 6);
  void* f[6] = {};
  for (int i = 0; x.ok && i < 6; ++i) f[i] = x.address(i);
  if (!x.ok) {
    PyErr_SetString(PyExc_ValueError, "six addresses expected");
    return nullptr;
  }
  f_append = reinterpret_cast<decltype(f_append)>(f[0]);
  f_attention = reinterpret_cast<decltype(f_attention)>(f[1]);
  f_tables_grow = reinterpret_cast<decltype(f_tables_grow)>(f[2]);
  f_rope_append = reinterpret_cast<decltype(f_rope_append)>(f[3]);
  f_prompt = reinterpret_cast<decltype(f_prompt)>(f[4]);
  f_read = reinterpret_cast<decltype(f_read)>(f[5]);
  Py_RETURN_NONE;
}

// No C++ exception crosses into Python: such a call goes the long way as well.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (...) {
    Py_RETURN_NONE;
  }
}

#define PA_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<name>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {PA_METHOD(append_kv),   PA_METHOD(attention),        PA_METHOD(tables_grow),
                         PA_METHOD(rope_append), PA_METHOD(prompt_attention), PA_METHOD(read_kv),
                         PA_METHOD(bind),        {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pa_bind() { return PyModule_Create(&module); }
