// Python binding of the serving calls (the ones made once per token and layer): takes the tensors'
// pointers, sizes and strides, the current stream and device straight from torch, makes the outputs
// that are not given, and calls the C entries of libsparge.so.  Nothing is computed here.  Through
// ctypes the same calls spend 17 to 34 us on the host, about twice what their kernels take at
// decoding sizes; here 4 to 8 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/sparge.h"

namespace {

PyObject *g_error = nullptr;  // the package's SpargeError

struct PyFail {};  // a Python exception is set

[[noreturn]] void type_error(const char *fmt, const char *name) {
  PyErr_Format(PyExc_TypeError, fmt, name);
  throw PyFail{};
}

// f() while other Python threads run: what may wait for the GPU (an allocation that frees others first, a launch into a full
// queue) belongs there.  f touches no Python object and raises no PyFail: a call's arguments are read and checked before.
// (One such stretch per call: each takes a few tenths of a microsecond.)
template <typename F>
auto unlocked(F f) {
  struct Unlock {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlock() { PyEval_RestoreThread(state); }
  } u;
  return f();
}

// The call's arguments after `self`, by position.
struct Args {
  PyObject *const *v;
  const char *call;
  Args(PyObject *const *v_, Py_ssize_t n, Py_ssize_t want, const char *call_) : v(v_), call(call_) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", call, want, n);
      throw PyFail{};
    }
  }
  bool none(int i) const { return v[i] == Py_None; }
  const at::Tensor &tensor(int i, const char *name) const {
    if (!THPVariable_Check(v[i])) type_error("%s must be a CUDA tensor", name);
    return THPVariable_Unpack(v[i]);
  }
  int64_t integer(int i) const {
    PyObject *x = PyNumber_Index(v[i]);
    if (!x) throw PyFail{};
    const int64_t r = PyLong_AsLongLong(x);
    Py_DECREF(x);
    if (r == -1 && PyErr_Occurred()) throw PyFail{};
    return r;
  }
  int small(int i) const {  // an int argument of the C entry
    const int64_t r = integer(i);
    return r > INT32_MAX ? INT32_MAX : r < INT32_MIN ? INT32_MIN : static_cast<int>(r);
  }
  float real(int i) const {
    const double r = PyFloat_AsDouble(v[i]);
    if (r == -1.0 && PyErr_Occurred()) throw PyFail{};
    return static_cast<float>(r);
  }
  bool truth(int i) const {
    const int r = PyObject_IsTrue(v[i]);
    if (r < 0) throw PyFail{};
    return r != 0;
  }
};

// The device of a call's first tensor, which has to be the current one: the kernels run there, on
// its current stream.
struct Here {
  int dev;
  cudaStream_t stream;
  explicit Here(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) {
      PyErr_Format(PyExc_ValueError, "%s is not on a CUDA device", name);
      throw PyFail{};
    }
    dev = c10::cuda::current_device();
    check(t, name);
    stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  }
  void check(const at::Tensor &t, const char *name) const {
    if (!t.is_cuda() || t.get_device() != dev) {
      PyErr_Format(PyExc_ValueError, "%s is on %s, the current CUDA device is cuda:%d", name, t.device().str().c_str(), dev);
      throw PyFail{};
    }
  }
  sparge_stream_t s() const { return reinterpret_cast<sparge_stream_t>(stream); }
  // a bf16 (B, H, N, d) tensor
  sparge_tensor rows(const at::Tensor &t, const char *name) const {
    check(t, name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 4 || t.stride(3) != 1)
      type_error("%s: expected a bf16 (B, H, N, d) tensor with contiguous last dim", name);
    return describe(t);
  }
  static sparge_tensor describe(const at::Tensor &t) {
    return sparge_tensor{t.data_ptr(), SPARGE_BF16, 0, t.size(0), t.size(1), t.size(2), t.size(3),
                         t.stride(0),  t.stride(1), t.stride(2)};
  }
  // a contiguous array of the given type and sizes (none: any)
  void *array(const at::Tensor &t, at::ScalarType type, const char *name, at::IntArrayRef shape) const {
    check(t, name);
    if (t.scalar_type() != type || !t.is_contiguous() || (!shape.empty() && t.sizes() != shape)) {
      PyErr_Format(PyExc_TypeError, "%s must be a contiguous %s tensor%s", name, at::toString(type),
                   shape.empty() ? "" : " of the shape that goes with the others");
      throw PyFail{};
    }
    return t.data_ptr();
  }
  sparge_cache4 pool(const at::Tensor &t) const {
    check(t, "pool");
    if (t.scalar_type() != at::kByte || t.dim() != 4 || !t.is_contiguous() || t.size(3) % 18 || t.size(1) > INT32_MAX ||
        t.size(2) > INT32_MAX / 16 || t.size(3) > INT32_MAX)
      type_error("%s must be a contiguous uint8 tensor of shape (n_pages, H, page_size / 16, 18 d)", "pool");
    return sparge_cache4{t.data_ptr(), t.size(0), static_cast<int32_t>(16 * t.size(2)), static_cast<int32_t>(t.size(1)),
                         static_cast<int32_t>(t.size(3) / 18), 0};
  }
  // an int32 (rows, width) page table: its stride between rows
  int64_t table(const at::Tensor &t, int64_t rows) const {
    check(t, "table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != rows || (t.size(1) > 1 && t.stride(1) != 1))
      type_error("%s must be an int32 tensor of one row per request, with contiguous rows", "table");
    return rows > 1 ? t.stride(0) : t.size(1);
  }
  // new tensors from torch's caching allocator, past the dispatcher (half of an empty()'s host time)
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt));
  }
  // a tensor of its own over a part of block's memory, `at` bytes in (several small outputs in one allocation)
  static at::Tensor part(const at::Tensor &block, int64_t at, at::IntArrayRef shape, at::ScalarType type) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(block.storage()), block.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    c10::TensorImpl *i = t.unsafeGetTensorImpl();
    i->set_sizes_contiguous(shape);
    i->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(type)));
    return t;
  }
  // like t: its strides where they leave no gaps, else contiguous
  at::Tensor make_like(const at::Tensor &t) const {
    if (t.is_contiguous() || !t.is_non_overlapping_and_dense()) return make(t.sizes(), t.scalar_type());
    return at::Tensor(at::detail::empty_strided_cuda(t.sizes(), t.strides(), t.scalar_type(),
                                                     at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev))));
  }
};

void done(int rc) {
  if (rc == SPARGE_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", rc, sparge_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw PyFail{};
}

PyObject *wrap(const at::Tensor &t) {
  PyObject *r = THPVariable_Wrap(t);
  if (!r) throw PyFail{};
  return r;
}

// A given tensor as it came (a new reference), else the one that was made.
PyObject *result(const Args &a, int i, const at::Tensor &t) {
  if (a.none(i)) return wrap(t);
  Py_INCREF(a.v[i]);
  return a.v[i];
}

template <typename... T>
PyObject *tuple_of(T... o) {
  PyObject *r = PyTuple_New(sizeof...(o));
  if (!r) {
    (Py_DECREF(o), ...);
    throw PyFail{};
  }
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, o), ...);
  return r;
}

// Argument i, a bf16 (B, H, N, d) tensor, or an undefined tensor for None.
at::Tensor given_rows(const Args &a, int i, const Here &h, const char *name) {
  if (a.none(i)) return {};
  h.rows(a.tensor(i, name), name);
  return a.tensor(i, name);
}
at::Tensor given_workspace(const Args &a, int i, const Here &h) {
  if (a.none(i)) return {};
  const at::Tensor &t = a.tensor(i, "ws");
  h.check(t, "ws");
  if (!t.is_contiguous()) type_error("%s must be contiguous", "ws");
  return t;
}
at::Tensor make_workspace(const Here &h, size_t bytes) { return h.make({static_cast<int64_t>(bytes ? bytes : 1)}, at::kByte); }

// (q, k, v, window, sinks, scale, out, ws)
PyObject *window_attn(const Args &a) {
  const at::Tensor &q = a.tensor(0, "q"), &k = a.tensor(1, "k"), &v = a.tensor(2, "v");
  const Here h(q, "q");
  const sparge_tensor dq = h.rows(q, "q"), dk = h.rows(k, "k"), dv = h.rows(v, "v");
  const int64_t window = a.integer(3), sinks = a.integer(4);
  const float scale = a.real(5);
  at::Tensor out = given_rows(a, 6, h, "out"), ws = given_workspace(a, 7, h);
  done(unlocked([&] {
    if (!out.defined()) out = h.make_like(q);
    if (!ws.defined()) ws = make_workspace(h, sparge_workspace_bytes(SPARGE_OP_WINDOW_ATTN, dk.B, dq.H, dk.H, dk.N, dk.d));
    sparge_tensor o = Here::describe(out);
    return sparge_window_attn(&dq, &dk, &dv, window, sinks, scale, &o, ws.data_ptr(), ws.nbytes(), h.s());
  }));
  return result(a, 6, out);
}

// (q, k, inv_freq, positions, start, q_weight, k_weight, eps, interleaved, q_out, k_out)
PyObject *qk_norm_rope(const Args &a) {
  const at::Tensor &q = a.tensor(0, "q"), &k = a.tensor(1, "k");
  const Here h(q, "q");
  const sparge_tensor dq = h.rows(q, "q"), dk = h.rows(k, "k");
  at::Tensor qo = given_rows(a, 9, h, "q_out"), ko = given_rows(a, 10, h, "k_out");
  const double *freq = nullptr;
  int64_t rot = 0;
  if (!a.none(2)) {
    const at::Tensor &f = a.tensor(2, "inv_freq");
    freq = static_cast<const double *>(h.array(f, at::kDouble, "inv_freq", {}));
    rot = 2 * f.numel();
  }
  const void *pos = a.none(3) ? nullptr : h.array(a.tensor(3, "positions"), at::kInt, "positions", {dq.B, dq.N});
  const void *w[2];
  for (int i = 0; i < 2; ++i)
    w[i] = a.none(5 + i) ? nullptr : h.array(a.tensor(5 + i, "weight"), at::kFloat, i ? "k_weight" : "q_weight", {dq.d});
  const int64_t start = a.integer(4);
  const float eps = a.real(7);
  const bool interleaved = a.truth(8);
  done(unlocked([&] {
    // small outputs share one allocation (64 tokens of 32 + 8 heads: 4.0 us of host time, 3.6 so); large ones do not, so that
    // letting go of one frees it
    const int64_t nq = static_cast<int64_t>(q.nbytes()), nk = static_cast<int64_t>(k.nbytes()), k0 = (nq + 255) / 256 * 256;
    if (!qo.defined() && !ko.defined() && nq + nk <= (1 << 20) && q.is_contiguous() && k.is_contiguous()) {
      const at::Tensor block = h.make({k0 + nk}, at::kByte);
      qo = Here::part(block, 0, q.sizes(), at::kBFloat16);
      ko = Here::part(block, k0, k.sizes(), at::kBFloat16);
    }
    if (!qo.defined()) qo = h.make_like(q);
    if (!ko.defined()) ko = h.make_like(k);
    sparge_tensor eq = Here::describe(qo), ek = Here::describe(ko);
    return sparge_qk_norm_rope(&dq, &dk, static_cast<const int32_t *>(pos), start, freq,
                               static_cast<int>(rot > INT32_MAX ? INT32_MAX : rot), interleaved, static_cast<const float *>(w[0]),
                               static_cast<const float *>(w[1]), eps, &eq, &ek, h.s());
  }));
  PyObject *r = result(a, 9, qo);
  return tuple_of(r, result(a, 10, ko));
}

// (lens, new_lens, free_pages, table, page_size, N, slots, positions, kv_lens, used)
PyObject *cache_tables(const Args &a) {
  const at::Tensor &lens = a.tensor(0, "lens"), &add = a.tensor(1, "new_lens"), &free = a.tensor(2, "free_pages"),
                   &table = a.tensor(3, "table");
  const Here h(lens, "lens");
  const int64_t R = lens.numel(), N = a.integer(5);
  const int page = a.small(4);
  if (N < 0 || N > (int64_t(1) << 30) || R > 65535) {
    PyErr_SetString(PyExc_ValueError, "N must be in 0..2^30, the requests at most 65535");
    throw PyFail{};
  }
  const auto i32 = [&](const at::Tensor &t, const char *name, at::IntArrayRef shape) {
    return static_cast<int32_t *>(h.array(t, at::kInt, name, shape));
  };
  const auto given = [&](int i, at::ScalarType type, const char *name, at::IntArrayRef shape) {
    if (a.none(i)) return at::Tensor();
    h.array(a.tensor(i, name), type, name, shape);
    return a.tensor(i, name);
  };
  const int32_t *pl = i32(lens, "lens", {R}), *pa = i32(add, "new_lens", {R}), *pf = i32(free, "free_pages", {});
  const int64_t stride = h.table(table, R);
  at::Tensor slots = given(6, at::kLong, "slots", {R, N}), pos = given(7, at::kInt, "positions", {R, N}),
             kv = given(8, at::kInt, "kv_lens", {R}), used = given(9, at::kInt, "used", {1});
  done(unlocked([&] {
    // small outputs share one allocation (four of them take the host longer than the kernel the GPU); large ones do not: the
    // lengths are kept for the next step, and would keep the slots and positions of this one
    const int64_t bs = slots.defined() ? 0 : 8 * R * N, bp = pos.defined() ? 0 : 4 * R * N, bk = kv.defined() ? 0 : 4 * R,
                  bu = used.defined() ? 0 : 4;
    const bool share = bs + bp + bk + bu <= (1 << 16);
    const bool any = !slots.defined() || !pos.defined() || !kv.defined() || !used.defined();
    const at::Tensor block = share && any ? h.make({bs + bp + bk + bu}, at::kByte) : at::Tensor();
    const auto made = [&](int64_t at, at::IntArrayRef shape, at::ScalarType type) {
      return share ? Here::part(block, at, shape, type) : h.make(shape, type);
    };
    if (!slots.defined()) slots = made(0, {R, N}, at::kLong);
    if (!pos.defined()) pos = made(bs, {R, N}, at::kInt);
    if (!kv.defined()) kv = made(bs + bp, {R}, at::kInt);
    if (!used.defined()) used = made(bs + bp + bk, {1}, at::kInt);
    return sparge_cache_tables(pl, pa, R, N, page, pf, free.numel(), static_cast<int32_t *>(table.data_ptr()), table.size(1), stride,
                               static_cast<int64_t *>(slots.data_ptr()), static_cast<int32_t *>(pos.data_ptr()),
                               static_cast<int32_t *>(kv.data_ptr()), static_cast<int32_t *>(used.data_ptr()), h.s());
  }));
  PyObject *r0 = result(a, 6, slots), *r1 = result(a, 7, pos), *r2 = result(a, 8, kv);
  return tuple_of(r0, r1, r2, result(a, 9, used));
}

// (k, v, slots, pool)
PyObject *cache4_store(const Args &a) {
  const at::Tensor &k = a.tensor(0, "k"), &v = a.tensor(1, "v");
  const Here h(k, "k");
  const sparge_tensor dk = h.rows(k, "k"), dv = h.rows(v, "v");
  const sparge_cache4 c = h.pool(a.tensor(3, "pool"));
  const int64_t *slots = static_cast<int64_t *>(h.array(a.tensor(2, "slots"), at::kLong, "slots", {dk.B, dk.N}));
  done(unlocked([&] { return sparge_cache4_store(&dk, &dv, slots, &c, h.s()); }));
  Py_RETURN_NONE;
}

// (pool, slots, k_out, v_out)
PyObject *cache4_load(const Args &a) {
  const at::Tensor &pool = a.tensor(0, "pool"), &slots = a.tensor(1, "slots");
  const Here h(pool, "pool");
  const sparge_cache4 c = h.pool(pool);
  if (a.none(2) != a.none(3)) {
    PyErr_SetString(PyExc_ValueError, "k_out and v_out are given together");
    throw PyFail{};
  }
  const bool made = a.none(2);
  if (slots.dim() != 2) type_error("%s must be a contiguous int64 (B, N) tensor", "slots");
  at::Tensor k = given_rows(a, 2, h, "k_out"), v = given_rows(a, 3, h, "v_out");
  const int64_t shape[4] = {made ? slots.size(0) : k.size(0), c.H, made ? slots.size(1) : k.size(2), c.d};
  const int64_t *where = static_cast<int64_t *>(h.array(slots, at::kLong, "slots", {shape[0], shape[2]}));
  done(unlocked([&] {
    const int64_t bytes = 2 * slots.numel() * c.H * c.d;
    if (made && bytes <= (1 << 19)) {  // small outputs share one allocation, as those of qk_norm_rope
      const at::Tensor block = h.make({2 * bytes}, at::kByte);
      k = Here::part(block, 0, shape, at::kBFloat16);
      v = Here::part(block, bytes, shape, at::kBFloat16);
    } else if (made) {
      k = h.make(shape, at::kBFloat16);
      v = h.make(shape, at::kBFloat16);
    }
    sparge_tensor dk = Here::describe(k), dv = Here::describe(v);
    return sparge_cache4_load(&c, where, made, &dk, &dv, h.s());
  }));
  PyObject *r = result(a, 2, k);
  return tuple_of(r, result(a, 3, v));
}

// (q, pool, table, kv_lens, window, sinks, scale, out, ws)
PyObject *cache4_attn(const Args &a) {
  const at::Tensor &q = a.tensor(0, "q"), &table = a.tensor(2, "table");
  const Here h(q, "q");
  const sparge_tensor dq = h.rows(q, "q");
  const sparge_cache4 c = h.pool(a.tensor(1, "pool"));
  const int64_t stride = h.table(table, dq.B);
  const int32_t *lens = static_cast<int32_t *>(h.array(a.tensor(3, "kv_lens"), at::kInt, "kv_lens", {dq.B}));
  const int64_t window = a.integer(4), sinks = a.integer(5);
  const float scale = a.real(6);
  at::Tensor out = given_rows(a, 7, h, "out"), ws = given_workspace(a, 8, h);
  done(unlocked([&] {
    if (!out.defined()) out = h.make_like(q);
    if (!ws.defined()) ws = make_workspace(h, sparge_cache4_attn_workspace_bytes(dq.B, dq.H, c.H, dq.N, dq.d));
    sparge_tensor o = Here::describe(out);
    return sparge_cache4_attn(&dq, &c, static_cast<const int32_t *>(table.data_ptr()), table.size(1), stride, lens, window, sinks,
                              scale, &o, ws.data_ptr(), ws.nbytes(), h.s());
  }));
  return result(a, 7, out);
}

// No C++ exception leaves through Python.
template <PyObject *(*F)(const Args &), int N>
PyObject *entry(PyObject *, PyObject *const *v, Py_ssize_t n) {
  try {
    return F(Args(v, n, N, "call"));
  } catch (const PyFail &) {
  } catch (const c10::OutOfMemoryError &e) {  // torch's own exception for it
    if (PyObject *torch = PyImport_ImportModule("torch")) {
      if (PyObject *cls = PyObject_GetAttrString(torch, "OutOfMemoryError")) {
        PyErr_SetString(cls, e.what_without_backtrace());
        Py_DECREF(cls);
      }
      Py_DECREF(torch);
    }
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject *set_error(PyObject *, PyObject *cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(window_attn, 8),
                         ENTRY(qk_norm_rope, 11),
                         ENTRY(cache_tables, 10),
                         ENTRY(cache4_store, 4),
                         ENTRY(cache4_load, 4),
                         ENTRY(cache4_attn, 9),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

extern "C" PyObject *PyInit__binding() { return PyModule_Create(&module); }
