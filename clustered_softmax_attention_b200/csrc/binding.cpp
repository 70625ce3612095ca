// CPython binding of the serving entry points (muse.py: muse_rope_axes, muse_cache_write,
// muse_cache_read, muse_cache_attend).
//
// These are called once a token and layer, on kernels of a few microseconds: marshalling them
// through Python objects takes longer than they run (13 us a call through ctypes, 5 here).
// Argument checks and marshalling only; each function returns its tensors, or the muse_status as
// an int when the library refused the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <stdexcept>
#include <string>

#include "muse.h"

namespace {

using at::Tensor;

struct Refused : std::invalid_argument {
  using std::invalid_argument::invalid_argument;
};

std::string say(const char *s) { return s; }
std::string say(int64_t v) { return std::to_string(v); }
std::string say(int v) { return std::to_string(v); }
std::string say(at::ScalarType t) { return at::toString(t); }
std::string say(at::Device d) { return d.str(); }
std::string say(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}
template <typename... A>
[[noreturn]] void refuse(const char *name, const A &...a) {
  std::string s = std::string(name) + ": ";
  ((s += say(a)), ...);
  throw Refused(s);
}

// A tensor argument; an undefined tensor for None.
Tensor take(PyObject *o, const char *name, bool optional = false) {
  if (optional && o == Py_None) return Tensor();
  if (!THPVariable_Check(o)) refuse(name, "expected a tensor");
  return THPVariable_Unpack(o);
}
int64_t whole(PyObject *o, const char *name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, "expected an integer");
  }
  return v;
}
double real(PyObject *o, const char *name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, "expected a number");
  }
  return v;
}
int small(int64_t v, const char *name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(name, "size ", v, " does not fit");
  return (int)v;
}

// The tensor that the others go by: four dimensions of float32 or bfloat16.
struct First {
  int B, H, N, D, dtype;
  at::ScalarType type;
  at::Device device;
};
First first(const Tensor &t, const char *name) {
  const auto type = t.scalar_type();
  if (t.dim() != 4 || (type != at::kFloat && type != at::kBFloat16))
    refuse(name, "expected float32 or bfloat16 with four dimensions, got ", type, " ", t.sizes());
  return {small(t.size(0), name), small(t.size(1), name), small(t.size(2), name), small(t.size(3), name),
          type == at::kFloat ? (int)MUSE_F32 : (int)MUSE_BF16, type, t.device()};
}
void same(const Tensor &t, const char *name, at::IntArrayRef shape, const First &f) {
  if (t.sizes() != shape) refuse(name, "shape ", t.sizes(), ", expected ", shape);
  if (t.scalar_type() != f.type || t.device() != f.device)
    refuse(name, t.scalar_type(), " on ", t.device(), ", expected ", f.type, " on ", f.device);
}

// Rows [B,H,N,D] as they lie; a dimension of size 1 has no stride of its own.
muse_rows rows(const Tensor &t, const char *name, bool written = false) {
  const auto n = t.sizes(), s = t.strides();
  const int64_t st[3] = {n[0] > 1 ? s[0] : 0, n[1] > 1 ? s[1] : 0, n[2] > 1 ? s[2] : 0};
  void *p = t.numel() ? t.data_ptr() : nullptr;
  const int64_t unit = 16 / t.element_size();
  if (s[3] != 1 || st[0] % unit || st[1] % unit || st[2] % unit || (uintptr_t)p % 16)
    refuse(name, "rows must be dense and 16-byte aligned, strides ", s);
  if (written) {
    // rows that are written must not overlap: each stride clears what is below it
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return st[a] < st[b]; });
    int64_t end = n[3];
    for (int i : order) {
      if (n[i] <= 1) continue;
      if (st[i] < end) refuse(name, "overlapping rows, strides ", s);
      end += st[i] * (n[i] - 1);
    }
  }
  if (!t.is_cuda()) refuse(name, "expected a CUDA tensor");
  return {p, st[0], st[1], st[2]};
}

const int32_t *ints(const Tensor &t, const char *name, at::IntArrayRef shape, at::Device device) {
  if (!t.defined()) return nullptr;
  if (t.sizes() != shape || t.scalar_type() != at::kInt || !t.is_contiguous() || t.device() != device)
    refuse(name, "expected a contiguous int32 tensor ", shape, " on ", device, ", got ",
           t.scalar_type(), " ", t.sizes(), " on ", t.device());
  return t.data_ptr<int32_t>();
}

struct Cache {
  muse_cache c;
  int Dv;
};
Cache cache_of(const Tensor &t, const Tensor &table, int64_t B, int64_t D, at::Device device) {
  if (t.dim() != 4 || t.scalar_type() != at::kByte || !t.is_contiguous() || t.device() != device)
    refuse("cache", "expected a contiguous uint8 tensor [pages,Hkv,page/32,bytes] on ", device, ", got ",
           t.scalar_type(), " ", t.sizes(), " on ", t.device());
  if (table.dim() != 2) refuse("page_table", "expected [B,max_pages], got ", table.sizes());
  const int64_t size = t.size(3), Dv = size / 18 - D, slots = table.size(1);
  if (size % 18 || (D != 64 && D != 128) || (Dv != 64 && Dv != 128))
    refuse("cache", "tiles of ", size, " bytes do not hold keys of width ", D);
  if (t.size(2) > 1 << 20) refuse("cache", "pages of ", t.size(2) * 32, " tokens");
  Cache r;
  r.c = {t.numel() ? t.data_ptr() : nullptr, ints(table, "page_table", {B, slots}, device),
         small(t.size(0), "cache"), small(t.size(1), "cache"), (int)t.size(2) * 32,
         small(slots, "page_table")};
  r.Dv = (int)Dv;
  return r;
}

Tensor made(at::IntArrayRef shape, at::ScalarType type, at::Device device, bool zero) {
  const auto o = at::TensorOptions().dtype(type).device(device);
  return zero ? at::zeros(shape, o) : at::empty(shape, o);
}
muse_stream_t stream(at::Device d) {
  return reinterpret_cast<muse_stream_t>(c10::cuda::getCurrentCUDAStream(d.index()).stream());
}

PyObject *pair(const Tensor &a, const Tensor &b) {
  PyObject *x = THPVariable_Wrap(a), *y = x ? THPVariable_Wrap(b) : nullptr;
  PyObject *t = y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

// (Q, positions, sections, base, K, flags, out, k_out)
PyObject *rope_axes(PyObject *const *a) {
  const Tensor Q = take(a[0], "Q"), pos = take(a[1], "positions");
  const First f = first(Q, "Q");
  muse_rope r = {};
  PyObject *seq = PySequence_Fast(a[2], "sections: expected a sequence of integers");
  if (!seq) return nullptr;
  const Py_ssize_t axes = PySequence_Fast_GET_SIZE(seq);
  try {
    if (axes < 1 || axes > MUSE_ROPE_MAX_AXES) refuse("sections", "1 to 4 axes, got ", (int64_t)axes);
    for (Py_ssize_t i = 0; i < axes; ++i)
      r.sections[i] = small(whole(PySequence_Fast_GET_ITEM(seq, i), "sections"), "sections");
  } catch (...) {
    Py_DECREF(seq);
    throw;
  }
  Py_DECREF(seq);
  r.axes = (int)axes;
  r.base = real(a[3], "base");
  const int64_t flags = whole(a[5], "flags");
  if (flags < 0 || flags > (int64_t)UINT32_MAX) refuse("flags", "unknown flags ", flags);
  r.flags = (unsigned)flags;
  const bool shared = pos.dim() == 2;
  const int32_t *p = shared ? ints(pos, "positions", {axes, f.N}, f.device)
                            : ints(pos, "positions", {f.B, axes, f.N}, f.device);
  const Tensor K = take(a[4], "K", true);
  auto place = [&](PyObject *o, const char *name, const Tensor &x) {
    Tensor y = take(o, name, true);
    if (!y.defined()) return made(x.sizes(), f.type, f.device, false);
    same(y, name, x.sizes(), f);
    if (y.data_ptr() == x.data_ptr() && y.strides() != x.strides())
      refuse(name, "in place needs the strides of its input");
    return y;
  };
  int Hk = 0;
  if (K.defined()) {
    if (K.dim() != 4) refuse("K", "shape ", K.sizes());
    Hk = small(K.size(1), "K");
    same(K, "K", {f.B, Hk, f.N, f.D}, f);
  }
  if (!Q.is_cuda()) {  // before anything is made there
    if (a[6] != Py_None) place(a[6], "out", Q);
    refuse("Q", "expected a CUDA tensor");
  }
  const c10::cuda::CUDAGuard guard(f.device);
  const Tensor out = place(a[6], "out", Q), k_out = K.defined() ? place(a[7], "k_out", K) : Tensor();
  const muse_rows none = {};
  const muse_rows q = rows(Q, "Q"), qo = rows(out, "out", true);
  const muse_rows k = K.defined() ? rows(K, "K") : none,
                  ko = K.defined() ? rows(k_out, "k_out", true) : none;
  const muse_dims d = {f.B, f.H, f.N, f.D, f.D, f.dtype, 1.0f};
  const muse_status s = muse_rope_axes(q, k, Hk, d, p, shared ? 1 : f.B, r, qo, ko, stream(f.device));
  if (s != MUSE_OK) return PyLong_FromLong(s);
  return K.defined() ? pair(out, k_out) : THPVariable_Wrap(out);
}

// (cache, K, V, page_table, start, counts)
PyObject *cache_write(PyObject *const *a) {
  const Tensor cache = take(a[0], "cache"), K = take(a[1], "K"), V = take(a[2], "V"),
               table = take(a[3], "page_table"), start = take(a[4], "start"),
               counts = take(a[5], "counts", true);
  const First f = first(K, "K");
  const Cache c = cache_of(cache, table, f.B, f.D, f.device);
  if (f.H != c.c.Hkv) refuse("K", "shape ", K.sizes(), ", the cache has ", c.c.Hkv, " heads");
  same(V, "V", {f.B, f.H, f.N, c.Dv}, f);
  const muse_rows k = rows(K, "K"), v = rows(V, "V");
  const int32_t *s0 = ints(start, "start", {f.B}, f.device), *n = ints(counts, "counts", {f.B}, f.device);
  const c10::cuda::CUDAGuard guard(f.device);
  const muse_dims d = {f.B, f.H, f.N, f.D, c.Dv, f.dtype, 1.0f};
  const muse_status s = muse_cache_write(k, v, d, c.c, s0, n, stream(f.device));
  if (s != MUSE_OK) return PyLong_FromLong(s);
  Py_INCREF(a[0]);
  return a[0];
}

// (cache, page_table, start, N, D, float32?, counts, K, V)
PyObject *cache_read(PyObject *const *a) {
  const Tensor cache = take(a[0], "cache"), table = take(a[1], "page_table"),
               start = take(a[2], "start"), counts = take(a[6], "counts", true);
  const int64_t N = whole(a[3], "N"), D = whole(a[4], "D");
  const int64_t B = table.dim() ? table.size(0) : 0;
  const at::Device device = cache.device();
  const Cache c = cache_of(cache, table, B, D, device);
  Tensor K = take(a[7], "K", true), V = take(a[8], "V", true);
  First f{(int)B, c.c.Hkv, small(N, "N"), (int)D, 0, at::kFloat, device};
  f.type = K.defined() ? K.scalar_type() : PyObject_IsTrue(a[5]) ? at::kFloat : at::kBFloat16;
  if (f.type != at::kFloat && f.type != at::kBFloat16)
    refuse("K", "expected float32 or bfloat16, got ", f.type);
  f.dtype = f.type == at::kFloat ? (int)MUSE_F32 : (int)MUSE_BF16;
  const int32_t *s0 = ints(start, "start", {B}, device), *n = ints(counts, "counts", {B}, device);
  if (K.defined() || V.defined()) {
    if (!K.defined() || !V.defined()) refuse("out", "expected (K, V)");
    same(K, "K", {B, c.c.Hkv, N, D}, f);
    same(V, "V", {B, c.c.Hkv, N, c.Dv}, f);
  }
  if (!cache.is_cuda()) refuse("cache", "expected a CUDA tensor");
  if (N < 0) refuse("N", "expected a size, got ", N);
  const c10::cuda::CUDAGuard guard(device);
  if (!K.defined()) {
    K = made({B, c.c.Hkv, N, D}, f.type, device, counts.defined());
    V = made({B, c.c.Hkv, N, c.Dv}, f.type, device, counts.defined());
  }
  const muse_rows k = rows(K, "K", true), v = rows(V, "V", true);
  const muse_dims d = {f.B, f.H, f.N, f.D, c.Dv, f.dtype, 1.0f};
  const muse_status s = muse_cache_read(d, c.c, s0, n, k, v, stream(device));
  if (s != MUSE_OK) return PyLong_FromLong(s);
  return pair(K, V);
}

// (Q, cache, page_table, lens, counts, scale, out, lse, ws)
PyObject *cache_attend(PyObject *const *a) {
  const Tensor Q = take(a[0], "Q"), cache = take(a[1], "cache"), table = take(a[2], "page_table"),
               lens = take(a[3], "lens"), counts = take(a[4], "counts", true);
  Tensor out = take(a[6], "out", true), lse = take(a[7], "lse", true), ws = take(a[8], "ws", true);
  const First f = first(Q, "Q");
  const Cache c = cache_of(cache, table, f.B, f.D, f.device);
  if (out.defined()) same(out, "out", {f.B, f.H, f.N, c.Dv}, f);
  if (lse.defined() && (lse.sizes() != at::IntArrayRef({f.B, f.H, f.N}) || lse.scalar_type() != at::kFloat ||
                        !lse.is_contiguous() || lse.device() != f.device))
    refuse("lse", "expected a contiguous float32 tensor ", at::IntArrayRef({f.B, f.H, f.N}), " on ",
           f.device);
  if (ws.defined() && (ws.scalar_type() != at::kByte || !ws.is_contiguous() || ws.device() != f.device))
    refuse("ws", "expected a contiguous uint8 tensor on ", f.device);
  const muse_rows q = rows(Q, "Q");
  const int32_t *n = ints(lens, "lens", {f.B}, f.device), *m = ints(counts, "counts", {f.B}, f.device);
  const muse_dims d = {f.B, f.H, f.N, f.D, c.Dv, f.dtype, (float)real(a[5], "scale")};
  const c10::cuda::CUDAGuard guard(f.device);
  if (!ws.defined()) {
    const size_t need = muse_workspace_size("muse_cache_attend", d, c.c.Hkv, 0, 0, 0, 0);
    if (!need) return PyLong_FromLong(MUSE_ERR_SHAPE);
    ws = made({(int64_t)need}, at::kByte, f.device, false);
  }
  if (!out.defined()) out = made({f.B, f.H, f.N, c.Dv}, f.type, f.device, counts.defined());
  if (!lse.defined()) lse = made({f.B, f.H, f.N}, at::kFloat, f.device, counts.defined());
  const muse_status s = muse_cache_attend(q, d, c.c, n, m, rows(out, "out", true), lse.data_ptr<float>(),
                                          ws.data_ptr(), (size_t)ws.numel(), stream(f.device));
  if (s != MUSE_OK) return PyLong_FromLong(s);
  return pair(out, lse);
}

// No C++ exception leaves a function that Python calls.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError &e) {
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define ENTRY(f, n) {#f, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {ENTRY(rope_axes, 8), ENTRY(cache_write, 6), ENTRY(cache_read, 9),
                          ENTRY(cache_attend, 9), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&kModule); }
