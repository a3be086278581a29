// The calls that a server makes every step and layer, marshalled in C++: the
// same checks and the same library calls as the Python binding's, in 1 to 2 us
// of host time instead of 6 to 10 (the launch itself takes 3).
//
// Each function takes the tensors as they are and either makes the call, when
// everything is plainly right (dtypes, shapes, contiguous, one device that is
// the current one), or says "not plain" (-1) and has done nothing: the Python
// binding then goes its own way, where every check has its message.  So what is
// accepted, refused and raised is the binding's alone to say.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include "diffattn.h"

namespace {

constexpr long kNotPlain = -1;

// The library's entry points (of its release or its bounds-checked build).
decltype(&diffattn_paged_step) g_step = nullptr;
decltype(&diffattn_rope) g_rope = nullptr;
decltype(&diffattn_kv_append) g_append = nullptr;
decltype(&diffattn_extend) g_extend = nullptr;

// The arguments of one call.  `ok` turns false for good with the first thing
// that is not plain.
struct Args {
  PyObject* const* a;
  Py_ssize_t n;
  bool ok = true;
  int device = -1;

  Args(PyObject* const* args, Py_ssize_t count, Py_ssize_t want) : a(args), n(count) { ok = count == want; }
  bool none(int i) const { return a[i] == Py_None; }
  // Tensor i: exactly a tensor, contiguous, on the one device.
  const at::Tensor* tensor(int i, at::ScalarType type) {
    if (!ok || !THPVariable_CheckExact(a[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.is_cuda() || t.scalar_type() != type || !t.is_contiguous()) return fail();
    if (device < 0) device = t.get_device();
    return t.get_device() == device ? &t : fail();
  }
  // The same with a shape.
  const at::Tensor* tensor(int i, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor* t = tensor(i, type);
    return t && t->sizes() == shape ? t : fail();
  }
  long long integer(int i) {
    const long long v = ok && PyLong_Check(a[i]) ? PyLong_AsLongLong(a[i]) : (ok = false, 0);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  int integer32(int i) {
    const long long v = integer(i);
    if (v < INT32_MIN || v > INT32_MAX) ok = false;
    return static_cast<int>(v);
  }
  float number(int i) {
    const double v = PyFloat_AsDouble(a[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<float>(v);
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  // Whether the call can be made: a library is bound, and the tensors' device is the current one.
  bool ready() const { return ok && g_extend && device >= 0 && c10::cuda::current_device() == device; }
  cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

bool fits32(long long x) { return x >= 0 && x <= INT32_MAX; }

PyObject* status(long s) { return PyLong_FromLong(s); }

template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {  // (out of memory, say: the binding meets it again and raises it)
    return status(kNotPlain);
  }
}

// The interpreter is free while the library is called.  An object, so that an
// exception from the arguments (a tensor without storage has no data_ptr) takes
// the interpreter back on its way out.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};
#define WITHOUT_GIL(call) \
  int st;                 \
  {                       \
    NoGil free;           \
    st = (call);          \
  }

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  g_step = reinterpret_cast<decltype(g_step)>(p[0]);
  g_rope = reinterpret_cast<decltype(g_rope)>(p[1]);
  g_append = reinterpret_cast<decltype(g_append)>(p[2]);
  g_extend = reinterpret_cast<decltype(g_extend)>(p[3]);
  Py_RETURN_NONE;
}

// ctx_lens, new_lens, block_table, free_pages, pool, pool_out, page_size, T, cu_q, kv_lens, positions, slots, info;
// with cu_q None the five results are parts of one new allocation, and come back in a tuple.
PyObject* paged_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args x(a, n, 13);
    const at::Tensor* bt = x.ok ? x.tensor(2, at::kInt) : nullptr;
    if (!bt || bt->dim() != 2) return status(kNotPlain);
    const int64_t S = bt->size(0), width = bt->size(1);
    const at::Tensor *ctx = x.tensor(0, at::kInt, {S}), *nl = x.tensor(1, at::kInt, {S}), *ring = x.tensor(3, at::kInt),
                     *pool = x.tensor(4, at::kInt, {2}), *pool_out = x.tensor(5, at::kInt, {2});
    const int page = x.integer32(6), T = x.integer32(7);
    if (!x.ok || ring->dim() != 1 || T < 0 || !fits32(S) || !fits32(width) || !fits32(ring->numel()))
      return status(kNotPlain);
    const int64_t sizes[5] = {S + 1, S, T, T, 4};
    std::vector<at::Tensor> made;
    const at::Tensor* out[5];
    const bool fresh = x.none(8);
    for (int i = 9; fresh && i < 13; ++i)
      if (!x.none(i)) return status(kNotPlain);
    if (fresh) {
      if (!x.ready()) return status(kNotPlain);
      made = at::unsafe_split_with_sizes(at::empty({2 * S + 2 * static_cast<int64_t>(T) + 5}, ctx->options()), sizes);
      for (int i = 0; i < 5; ++i) out[i] = &made[i];
    } else {
      for (int i = 0; i < 5; ++i) out[i] = x.tensor(8 + i, at::kInt, {sizes[i]});
    }
    if (!x.ready()) return status(kNotPlain);
    auto p = [](const at::Tensor* t) { return static_cast<int*>(t->data_ptr()); };
    const cudaStream_t s = x.stream();
    WITHOUT_GIL(g_step(p(ctx), p(nl), static_cast<int>(S), p(bt), static_cast<int>(width), p(ring),
                       static_cast<int>(ring->numel()), p(pool), p(pool_out), page, T, p(out[0]), p(out[1]), p(out[2]),
                       p(out[3]), p(out[4]), s));
    if (st != 0 || !fresh) return status(st);
    PyObject* t = PyTuple_New(5);
    if (!t) return nullptr;
    for (int i = 0; i < 5; ++i) {
      PyObject* item = THPVariable_Wrap(made[i]);
      if (!item) {
        Py_DECREF(t);
        return nullptr;
      }
      PyTuple_SET_ITEM(t, i, item);
    }
    return t;
  });
}

// The rotation's table: (n_pos, rot), or false.
bool rotation(Args& x, int i_pos, int i_table, int64_t T, int64_t d, int* n_pos, int* rot, const at::Tensor** pos,
              const at::Tensor** table) {
  *pos = x.tensor(i_pos, at::kInt);
  *table = x.tensor(i_table, at::kFloat);
  if (!x.ok || (*pos)->numel() != T || (*table)->dim() != 3 || (*table)->size(2) != 2) return false;
  const int64_t np = (*table)->size(0), half = (*table)->size(1);
  if (np < 1 || half < 1 || half > d / 2 || !fits32(np)) return false;
  *n_pos = static_cast<int>(np);
  *rot = static_cast<int>(2 * half);
  return true;
}

// q, k (or None), positions, table, layout, inverse, q_out, k_out (or None)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args x(a, n, 8);
    if (!x.ok || !THPVariable_CheckExact(a[0])) return status(kNotPlain);
    const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) return status(kNotPlain);
    const at::Tensor* q = x.tensor(0, type);
    if (!q || q->dim() < 4 || q->size(-2) != 2) return status(kNotPlain);
    const int64_t nd = q->dim(), d = q->size(-1), H = q->size(-3);
    const int64_t T = q->sizes().slice(0, nd - 3).empty() ? 1 : c10::multiply_integers(q->sizes().slice(0, nd - 3));
    const at::Tensor *k = nullptr, *ko = nullptr;
    int64_t H_kv = 0;
    if (!x.none(1)) {
      k = x.tensor(1, type);
      if (!k || k->dim() != nd || k->size(-1) != d || k->size(-2) != 2 ||
          k->sizes().slice(0, nd - 3) != q->sizes().slice(0, nd - 3))
        return status(kNotPlain);
      H_kv = k->size(-3);
      ko = x.tensor(7, type, k->sizes());
    } else if (!x.none(7)) {
      return status(kNotPlain);
    }
    const at::Tensor* qo = x.tensor(6, type, q->sizes());
    const at::Tensor *pos, *table;
    int n_pos, rot;
    if (!rotation(x, 2, 3, T, d, &n_pos, &rot, &pos, &table)) return status(kNotPlain);
    const int layout = x.integer32(4), inverse = x.integer32(5);
    if (!x.ready() || !fits32(T) || !fits32(H) || !fits32(H_kv) || !fits32(d)) return status(kNotPlain);
    const cudaStream_t s = x.stream();
    WITHOUT_GIL(g_rope(q->data_ptr(), k ? k->data_ptr() : nullptr, static_cast<const int*>(pos->data_ptr()),
                       static_cast<const float*>(table->data_ptr()), n_pos, static_cast<int>(T), static_cast<int>(H),
                       static_cast<int>(H_kv), static_cast<int>(d), rot,
                       type == at::kBFloat16 ? DIFFATTN_BF16 : DIFFATTN_F32, layout, inverse, qo->data_ptr(),
                       ko ? ko->data_ptr() : nullptr, s));
    return status(st);
  });
}

// A paged cache: its tensors, and its sizes if q's heads are d wide.
bool cache(Args& x, int i_k, int i_v, int64_t d, const at::Tensor** kc, const at::Tensor** vc) {
  *kc = x.tensor(i_k, at::kBFloat16);
  if (!x.ok || (*kc)->dim() != 5 || (*kc)->size(3) != 2 || (*kc)->size(4) != d) return false;
  *vc = x.tensor(i_v, at::kBFloat16, {(*kc)->size(0), (*kc)->size(1), (*kc)->size(2), 2 * d});
  return x.ok && fits32((*kc)->size(0)) && fits32((*kc)->size(1)) && fits32((*kc)->size(2));
}

// q, k, v, positions, slots, table (or None), k_cache, v_cache, layout, q_out
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args x(a, n, 10);
    const at::Tensor* q = x.ok ? x.tensor(0, at::kBFloat16) : nullptr;
    if (!q || q->dim() != 4 || q->size(2) != 2) return status(kNotPlain);
    const int64_t T = q->size(0), H = q->size(1), d = q->size(3);
    const at::Tensor *kc, *vc, *pos = nullptr, *table = nullptr;
    if (!cache(x, 6, 7, d, &kc, &vc)) return status(kNotPlain);
    const int64_t H_kv = kc->size(2);
    const at::Tensor *k = x.tensor(1, at::kBFloat16, {T, H_kv, 2, d}), *v = x.tensor(2, at::kBFloat16, {T, H_kv, 2 * d}),
                     *slots = x.tensor(4, at::kInt, {T}), *out = x.tensor(9, at::kBFloat16, q->sizes());
    int n_pos = 0, rot = 0;
    if (!x.none(5) && !rotation(x, 3, 5, T, d, &n_pos, &rot, &pos, &table)) return status(kNotPlain);
    const int layout = x.integer32(8);
    if (!x.ready() || !fits32(T) || !fits32(H) || !fits32(d)) return status(kNotPlain);
    const cudaStream_t s = x.stream();
    WITHOUT_GIL(g_append(q->data_ptr(), k->data_ptr(), v->data_ptr(),
                         pos ? static_cast<const int*>(pos->data_ptr()) : nullptr,
                         static_cast<const int*>(slots->data_ptr()),
                         table ? static_cast<const float*>(table->data_ptr()) : nullptr, n_pos, static_cast<int>(T),
                         static_cast<int>(H), static_cast<int>(H_kv), static_cast<int>(d), rot, layout,
                         static_cast<int>(kc->size(0)), static_cast<int>(kc->size(1)), out->data_ptr(), kc->data_ptr(),
                         vc->data_ptr(), s));
    return status(st);
  });
}

// q, k_cache, v_cache, block_table, plan buffer, S, T, H, H_kv, d, max_new, lambda, lambda_init, rms_w, eps, mode,
// workspace, out
PyObject* extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args x(a, n, 18);
    if (!x.ok) return status(kNotPlain);
    const int S = x.integer32(5), T = x.integer32(6), H = x.integer32(7), H_kv = x.integer32(8), d = x.integer32(9),
              max_new = x.integer32(10), mode = x.integer32(15);
    const at::Tensor* q = x.tensor(0, at::kBFloat16, {T, H, 2, d});
    const at::Tensor *kc, *vc;
    if (!q || !cache(x, 1, 2, d, &kc, &vc) || kc->size(2) != H_kv) return status(kNotPlain);
    const at::Tensor *bt = x.tensor(3, at::kInt), *plan = x.tensor(4, at::kByte), *lam = x.tensor(11, at::kFloat),
                     *w = x.tensor(13, at::kFloat), *ws = x.tensor(16, at::kByte),
                     *out = x.tensor(17, at::kBFloat16, {T, H, 2 * static_cast<int64_t>(d)});
    const float lambda_init = x.number(12), eps = x.number(14);
    if (!x.ready() || bt->dim() != 2 || bt->size(0) != S || !fits32(bt->size(1)) || lam->numel() < 1 ||
        w->numel() != 2 * static_cast<int64_t>(d))
      return status(kNotPlain);
    const cudaStream_t s = x.stream();
    WITHOUT_GIL(g_extend(q->data_ptr(), kc->data_ptr(), vc->data_ptr(), static_cast<const int*>(bt->data_ptr()),
                         static_cast<int>(bt->size(1)), static_cast<int>(kc->size(0)), static_cast<int>(kc->size(1)),
                         plan->data_ptr(), plan->nbytes(), S, T, H, H_kv, d, max_new,
                         static_cast<const float*>(lam->data_ptr()), lambda_init,
                         static_cast<const float*>(w->data_ptr()), eps, mode, out->data_ptr(), ws->data_ptr(),
                         ws->nbytes(), s));
    return status(st);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<bind>("bind"),           method<paged_step>("paged_step"), method<rope>("rope"),
                           method<kv_append>("kv_append"), method<extend>("extend"),         {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
