// py_fast.cpp -- the short way from Python into the per-block entry points.
//
// A small decode step is paced by the host: checking eight tensors from Python
// and calling through ctypes takes 7 to 10 us, the kernels 3 to 5.  Each function
// here reads the tensors of one call in C++, makes the call when everything is as
// the call wants it, and returns True.  Whatever is not (a type, a shape, a
// stride, another device, a status) makes it return False with nothing launched;
// api.py then takes its own way, which names what is wrong.  So api.py defines the
// checks and the errors, and this file holds no message.
//
// Arguments after the tensors and numbers of the call: the current device and the
// stream's handle.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "pagedattn.h"

namespace {

// The library's entry points, handed over by api.py from the library it loaded.
decltype(&pa_reshape_and_cache_fp8_block) g_write;
decltype(&pa_update_key_bounds) g_bounds;
decltype(&pa_decode_fp8_block) g_decode;
decltype(&pa_decode_splitk_fp8_block) g_splitk;
decltype(&pa_prefill_fp8_block) g_prefill;
decltype(&pa_select_blocks) g_select;
decltype(&pa_decode_sparse) g_sparse;

constexpr int64_t kIntMax = 0x7fffffff;

// The arguments of one call, read in order; `ok` falls with the first that is not as wanted.
struct Args {
  PyObject* const* a;
  long device;
  bool ok = true;

  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : a(args), device(-1) {
    ok = n == want;
    if (ok) device = integer(static_cast<int>(n) - 2);
  }
  long integer(int i) {
    const long v = ok && PyLong_Check(a[i]) ? PyLong_AsLong(a[i]) : -1;
    if (v == -1) {
      ok = false;
      PyErr_Clear();
    }
    return v;
  }
  void* stream(int i) {
    void* s = ok && PyLong_Check(a[i]) ? PyLong_AsVoidPtr(a[i]) : nullptr;
    if (PyErr_Occurred()) {
      ok = false;
      PyErr_Clear();
    }
    return s;
  }
  float real(int i) {
    if (!ok || !PyFloat_Check(a[i])) {
      ok = false;
      return 0.f;
    }
    return static_cast<float>(PyFloat_AS_DOUBLE(a[i]));
  }
  // A contiguous CUDA tensor of the call's device.
  const at::Tensor* tensor(int i) {
    if (!ok || !THPVariable_Check(a[i])) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    ok = t.is_cuda() && t.get_device() == device && t.is_contiguous();
    return &t;
  }
  void* typed(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(i);
    ok = ok && t->scalar_type() == type && t->sizes() == c10::IntArrayRef(shape);
    return ok ? t->data_ptr() : nullptr;
  }
  void* codes(int i, c10::IntArrayRef shape) {
    const at::Tensor* t = tensor(i);
    ok = ok && (t->scalar_type() == at::kByte || t->scalar_type() == at::kFloat8_e4m3fn) && t->sizes() == shape;
    return ok ? t->data_ptr() : nullptr;
  }
};

int dtype_code(at::ScalarType t) { return t == at::kHalf ? PA_FP16 : t == at::kBFloat16 ? PA_BF16 : -1; }
bool fits(std::initializer_list<int64_t> v) {
  for (int64_t x : v)
    if (x > kIntMax) return false;
  return true;
}

PyObject* answer(bool done) { return PyBool_FromLong(done ? 1 : 0); }

#define PA_FAST(name) PyObject* name##_(PyObject*, PyObject* const* args, Py_ssize_t n) noexcept try
#define PA_GUARD catch (...) { return answer(false); }  // what a tensor's accessors throw: api.py says why

// One entry point's call, the interpreter free for other threads meanwhile.
template <class F, class... A>
PyObject* launch(F f, A... a) {
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = f(a...);
  Py_END_ALLOW_THREADS;
  return answer(status == PA_OK);
}

// key, value, k_cache, v_cache, k_scales, v_scales, slot_mapping
PA_FAST(write) {
  Args x(args, n, 9);
  const at::Tensor* key = x.tensor(0); const at::Tensor* pool = x.tensor(2);
  if (!x.ok || key->dim() != 3 || pool->dim() != 4) return answer(false);
  const int64_t T = key->size(0), N = pool->size(0), B = pool->size(1), Hk = pool->size(2), d = pool->size(3);
  const at::ScalarType dt = key->scalar_type(); const int code = dtype_code(dt);
  void* k = x.typed(0, dt, {T, Hk, d}); void* v = x.typed(1, dt, {T, Hk, d});
  void* kc = x.codes(2, pool->sizes()); void* vc = x.codes(3, pool->sizes());
  void* ks = x.typed(4, at::kFloat, {N, Hk}); void* vs = x.typed(5, at::kFloat, {N, Hk});
  void* sm = x.typed(6, at::kLong, {T}); void* st = x.stream(8);
  if (!x.ok || code < 0 || !fits({T, N, B, Hk, d})) return answer(false);
  return launch(g_write, k, v, kc, vc, static_cast<float*>(ks), static_cast<float*>(vs), static_cast<int64_t*>(sm), T, N,
                        B, Hk, d, code, st);
} PA_GUARD

// key, key_bounds, bound_exps, slot_mapping, block_size
PA_FAST(bounds) {
  Args x(args, n, 7);
  const at::Tensor* key = x.tensor(0); const at::Tensor* bd = x.tensor(1);
  if (!x.ok || key->dim() != 3 || bd->dim() != 4) return answer(false);
  const int64_t T = key->size(0), Hk = key->size(1), d = key->size(2), N = bd->size(0);
  const at::ScalarType dt = key->scalar_type(); const int code = dtype_code(dt);
  void* k = x.typed(0, dt, {T, Hk, d}); void* b = x.typed(1, at::kChar, {N, Hk, 2, d});
  void* e = x.typed(2, at::kInt, {N, Hk}); void* sm = x.typed(3, at::kLong, {T});
  const long B = x.integer(4); void* st = x.stream(6);
  if (!x.ok || code < 0 || !fits({T, N, B, Hk, d})) return answer(false);
  return launch(g_bounds, k, static_cast<int8_t*>(b), static_cast<int32_t*>(e), static_cast<int64_t*>(sm), T, N, B, Hk, d,
                         code, st);
} PA_GUARD

// out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale
PA_FAST(decode) {
  Args x(args, n, 11);
  const at::Tensor* q = x.tensor(1); const at::Tensor* pool = x.tensor(2); const at::Tensor* bt = x.tensor(6);
  if (!x.ok || q->dim() != 3 || pool->dim() != 4 || bt->dim() != 2) return answer(false);
  const int64_t S = q->size(0), H = q->size(1), d = q->size(2), N = pool->size(0), B = pool->size(1), Hk = pool->size(2);
  const int64_t M = bt->size(1); const at::ScalarType dt = q->scalar_type(); const int code = dtype_code(dt);
  void* o = x.typed(0, dt, {S, H, d}); void* qp = x.typed(1, dt, {S, H, d});
  void* kc = x.codes(2, pool->sizes()); void* vc = x.codes(3, pool->sizes());
  void* ks = x.typed(4, at::kFloat, {N, Hk}); void* vs = x.typed(5, at::kFloat, {N, Hk});
  void* tp = x.typed(6, at::kInt, {S, M}); void* cl = x.typed(7, at::kInt, {S});
  const float scale = x.real(8); void* st = x.stream(10);
  if (!x.ok || code < 0 || pool->size(3) != d || !fits({S, H, d, N, B, Hk, M})) return answer(false);
  return launch(g_decode, o, qp, kc, vc, static_cast<float*>(ks), static_cast<float*>(vs), static_cast<int32_t*>(tp), M,
                         static_cast<int32_t*>(cl), S, H, Hk, d, B, N, scale, code, st);
} PA_GUARD

// as decode, then partition_size, max_num_partitions, workspace
PA_FAST(splitk) {
  Args x(args, n, 14);
  const at::Tensor* q = x.tensor(1); const at::Tensor* pool = x.tensor(2); const at::Tensor* bt = x.tensor(6);
  const at::Tensor* ws = x.tensor(11);
  if (!x.ok || q->dim() != 3 || pool->dim() != 4 || bt->dim() != 2) return answer(false);
  const int64_t S = q->size(0), H = q->size(1), d = q->size(2), N = pool->size(0), B = pool->size(1), Hk = pool->size(2);
  const int64_t M = bt->size(1); const at::ScalarType dt = q->scalar_type(); const int code = dtype_code(dt);
  void* o = x.typed(0, dt, {S, H, d}); void* qp = x.typed(1, dt, {S, H, d});
  void* kc = x.codes(2, pool->sizes()); void* vc = x.codes(3, pool->sizes());
  void* ks = x.typed(4, at::kFloat, {N, Hk}); void* vs = x.typed(5, at::kFloat, {N, Hk});
  void* tp = x.typed(6, at::kInt, {S, M}); void* cl = x.typed(7, at::kInt, {S});
  const float scale = x.real(8); const long ps = x.integer(9), P = x.integer(10); void* st = x.stream(13);
  if (!x.ok || code < 0 || pool->size(3) != d || !fits({S, H, d, N, B, Hk, M, ps, P})) return answer(false);
  return launch(g_splitk, o, qp, kc, vc, static_cast<float*>(ks), static_cast<float*>(vs), static_cast<int32_t*>(tp), M,
                         static_cast<int32_t*>(cl), S, H, Hk, d, B, N, scale, code, ps, P, ws->data_ptr(), ws->nbytes(),
                         st);
} PA_GUARD

// out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, query_start_loc, max_query_len, scale
PA_FAST(prefill) {
  Args x(args, n, 13);
  const at::Tensor* q = x.tensor(1); const at::Tensor* pool = x.tensor(2); const at::Tensor* bt = x.tensor(6);
  if (!x.ok || q->dim() != 3 || pool->dim() != 4 || bt->dim() != 2) return answer(false);
  const int64_t R = q->size(0), H = q->size(1), d = q->size(2), N = pool->size(0), B = pool->size(1), Hk = pool->size(2);
  const int64_t S = bt->size(0), M = bt->size(1); const at::ScalarType dt = q->scalar_type();
  const int code = dtype_code(dt);
  void* o = x.typed(0, dt, {R, H, d}); void* qp = x.typed(1, dt, {R, H, d});
  void* kc = x.codes(2, pool->sizes()); void* vc = x.codes(3, pool->sizes());
  void* ks = x.typed(4, at::kFloat, {N, Hk}); void* vs = x.typed(5, at::kFloat, {N, Hk});
  void* tp = x.typed(6, at::kInt, {S, M}); void* cl = x.typed(7, at::kInt, {S}); void* qs = x.typed(8, at::kInt, {S + 1});
  const long maxq = x.integer(9); const float scale = x.real(10); void* st = x.stream(12);
  if (!x.ok || code < 0 || pool->size(3) != d || !fits({R, S, H, d, N, B, Hk, M, maxq})) return answer(false);
  return launch(g_prefill, o, qp, kc, vc, static_cast<float*>(ks), static_cast<float*>(vs), static_cast<int32_t*>(tp), M,
                          static_cast<int32_t*>(cl), static_cast<int32_t*>(qs), S, R, maxq, H, Hk, d, B, N, scale, code,
                          st);
} PA_GUARD

// sel_tables, sel_lens, q, key_bounds, bound_exps, block_tables, context_lens, block_size, num_first, num_last, workspace
PA_FAST(select) {
  Args x(args, n, 13);
  const at::Tensor* sel = x.tensor(0); const at::Tensor* q = x.tensor(2); const at::Tensor* bd = x.tensor(3);
  const at::Tensor* bt = x.tensor(5); const at::Tensor* ws = x.tensor(10);
  if (!x.ok || sel->dim() != 3 || q->dim() != 3 || bd->dim() != 4 || bt->dim() != 2) return answer(false);
  const int64_t S = q->size(0), H = q->size(1), d = q->size(2), Hk = sel->size(1), K = sel->size(2), N = bd->size(0);
  const int64_t M = bt->size(1); const at::ScalarType dt = q->scalar_type(); const int code = dtype_code(dt);
  void* tab = x.typed(0, at::kInt, {S, Hk, K}); void* len = x.typed(1, at::kInt, {S, Hk});
  void* qp = x.typed(2, dt, {S, H, d}); void* b = x.typed(3, at::kChar, {N, Hk, 2, d});
  void* e = x.typed(4, at::kInt, {N, Hk}); void* tp = x.typed(5, at::kInt, {S, M}); void* cl = x.typed(6, at::kInt, {S});
  const long B = x.integer(7), first = x.integer(8), last = x.integer(9); void* st = x.stream(12);
  if (!x.ok || code < 0 || !fits({S, H, d, Hk, K, N, M, B, first, last})) return answer(false);
  return launch(g_select, static_cast<int32_t*>(tab), static_cast<int32_t*>(len), qp, static_cast<int8_t*>(b),
                         static_cast<int32_t*>(e), static_cast<int32_t*>(tp), M, static_cast<int32_t*>(cl), S, H, Hk, d,
                         B, N, K, first, last, code, ws->data_ptr(), ws->nbytes(), st);
} PA_GUARD

// out, q, k_cache, v_cache, sel_tables, sel_lens, scale, k_scales or None, v_scales or None
PA_FAST(sparse) {
  Args x(args, n, 11);
  const at::Tensor* q = x.tensor(1); const at::Tensor* pool = x.tensor(2); const at::Tensor* sel = x.tensor(4);
  if (!x.ok || q->dim() != 3 || pool->dim() != 4 || sel->dim() != 3) return answer(false);
  const int64_t S = q->size(0), H = q->size(1), d = q->size(2), N = pool->size(0), B = pool->size(1), Hk = pool->size(2);
  const int64_t K = sel->size(2); const at::ScalarType dt = q->scalar_type(); const int code = dtype_code(dt);
  void* o = x.typed(0, dt, {S, H, d}); void* qp = x.typed(1, dt, {S, H, d});
  void* tab = x.typed(4, at::kInt, {S, Hk, K}); void* len = x.typed(5, at::kInt, {S, Hk});
  const float scale = x.real(6); void* st = x.stream(10);
  void* kc; void* vc; void* ks = nullptr; void* vs = nullptr; int kv = code;
  if (args[7] == Py_None && args[8] == Py_None) {
    kc = x.typed(2, dt, {N, B, Hk, d});
    vc = x.typed(3, dt, {N, B, Hk, d});
  } else {
    kc = x.codes(2, pool->sizes());
    vc = x.codes(3, pool->sizes());
    ks = x.typed(7, at::kFloat, {N, Hk});
    vs = x.typed(8, at::kFloat, {N, Hk});
    kv = PA_FP8_E4M3;
  }
  if (!x.ok || code < 0 || pool->size(3) != d || !fits({S, H, d, N, B, Hk, K})) return answer(false);
  return launch(g_sparse, o, qp, kc, vc, static_cast<float*>(ks), static_cast<float*>(vs), static_cast<int32_t*>(tab), K,
                         static_cast<int32_t*>(len), S, H, Hk, d, B, N, scale, code, kv, st);
} PA_GUARD

// bind(write, bounds, decode, splitk, prefill, select, sparse): the entry points' addresses
PyObject* bind_(PyObject*, PyObject* const* args, Py_ssize_t n) noexcept {
  void* p[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
      return nullptr;
    }
  }
  g_write = reinterpret_cast<decltype(g_write)>(p[0]);
  g_bounds = reinterpret_cast<decltype(g_bounds)>(p[1]);
  g_decode = reinterpret_cast<decltype(g_decode)>(p[2]);
  g_splitk = reinterpret_cast<decltype(g_splitk)>(p[3]);
  g_prefill = reinterpret_cast<decltype(g_prefill)>(p[4]);
  g_select = reinterpret_cast<decltype(g_select)>(p[5]);
  g_sparse = reinterpret_cast<decltype(g_sparse)>(p[6]);
  Py_RETURN_NONE;
}

#define PA_METHOD(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name##_)), METH_FASTCALL, nullptr }
PyMethodDef g_methods[] = {PA_METHOD(bind),    PA_METHOD(write),  PA_METHOD(bounds), PA_METHOD(decode), PA_METHOD(splitk),
                           PA_METHOD(prefill), PA_METHOD(select), PA_METHOD(sparse), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&g_module); }
