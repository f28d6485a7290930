// Python entry points of the handle-free attention operators (module _attention): argument checks,
// output and workspace memory, and the calls of include/dreamer.h, without a Python statement a
// check; a small call's time is its host time.  attention.py holds the interface and its
// documentation.  Every function returns its outputs, or the error code of the C entry point as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <math.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dreamer.h"

namespace {

constexpr int64_t ANY = -1;

// A refused argument: a Python ValueError, carried to the entry point
struct Refused {};
template <typename... A> [[noreturn]] void refuse(const char *fmt, A... a) {
  PyErr_Format(PyExc_ValueError, fmt, a...);
  throw Refused();
}

struct Rows {
  void *p;
  int64_t ld, n, h, d;
  int dtype;  // 0 float32, 1 bfloat16
};

const at::Tensor &tensor(const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) refuse("%s: a tensor", name);
  return THPVariable_Unpack(o);
}

// A tensor [rows][heads][dim] of device `dev` whose rows are 16-byte aligned and whose heads lie densely
Rows rows(const char *name, PyObject *o, int dev, int64_t heads = ANY, int64_t dim = ANY, int dtype = -1,
          int64_t n = ANY) {
  const at::Tensor &t = tensor(name, o);
  const auto st = t.scalar_type();
  if (!t.is_cuda() || t.get_device() != dev || t.dim() != 3 || (st != at::kFloat && st != at::kBFloat16))
    refuse("%s: a float32 or bfloat16 tensor [rows][heads][dim] on cuda:%d", name, dev);
  Rows r;
  r.n = t.size(0);
  r.h = t.size(1);
  r.d = t.size(2);
  r.dtype = st == at::kFloat ? 0 : 1;
  if ((heads != ANY && r.h != heads) || (dim != ANY && r.d != dim) || (n != ANY && r.n != n) ||
      (dtype >= 0 && r.dtype != dtype))
    refuse("%s: [%lld][%lld][%lld] of %s does not fit the other arguments", name, (long long)r.n, (long long)r.h,
           (long long)r.d, r.dtype ? "bfloat16" : "float32");
  const int64_t w = r.h * r.d, align = r.dtype ? 8 : 4;
  if (t.is_contiguous()) {
    r.ld = w;
  } else {
    r.ld = t.stride(0);
    if ((t.stride(2) != 1 && r.d > 1) || (t.stride(1) != r.d && r.h > 1) || (r.ld < w && r.n > 1))
      refuse("%s: a row's heads have to lie densely (strides %lld, %lld, %lld)", name, (long long)t.stride(0),
             (long long)t.stride(1), (long long)t.stride(2));
  }
  if (r.n <= 1) r.ld = (w + align - 1) / align * align;  // one row has no stride
  r.p = t.data_ptr();
  if ((r.n > 0 && ((uintptr_t)r.p & 15)) || r.ld % align) refuse("%s: rows have to be 16-byte aligned", name);
  return r;
}

// An output must not lie over an input; both may be columns of one buffer
void apart(const char *name, const Rows &o, const Rows &x) {
  if (o.n == 0 || x.n == 0) return;
  const int64_t es = o.dtype ? 2 : 4, wo = o.h * o.d, wx = x.h * x.d;
  const intptr_t o0 = (intptr_t)o.p, x0 = (intptr_t)x.p;
  if (o0 + ((o.n - 1) * o.ld + wo) * es <= x0 || x0 + ((x.n - 1) * x.ld + wx) * es <= o0) return;
  if (o.ld == x.ld && (x0 - o0) % es == 0) {
    const int64_t c = ((x0 - o0) / es % o.ld + o.ld) % o.ld;  // x's first column from out's
    if (c >= wo && c + wx <= o.ld) return;
  }
  refuse("out: overlaps %s", name);
}

int32_t *ints(const char *name, PyObject *o, int dev, int64_t n) {
  const at::Tensor &t = tensor(name, o);
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n ||
      !t.is_contiguous())
    refuse("%s: a contiguous int32 tensor of %lld on cuda:%d", name, (long long)n, dev);
  return t.data_ptr<int32_t>();
}

int32_t *status_of(PyObject *o, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor &t = tensor("status", o);
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kInt || t.numel() < 1)
    refuse("status: an int32 tensor on cuda:%d", dev);
  return t.data_ptr<int32_t>();
}

float scale_of(PyObject *o, int64_t d) {
  if (o == Py_None) return (float)(1.0 / sqrt((double)d));
  const double s = PyFloat_AsDouble(o);
  if (s == -1.0 && PyErr_Occurred()) throw Refused();
  if (!isfinite((float)s * 1.4426950408889634f)) refuse("scale: a number below 2.3e38");  // as the library
  return (float)s;
}

int64_t whole(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

// Memory and launches may wait for the device, whose host functions may want the interpreter
struct Unlocked {
  PyThreadState *st = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(st); }
};
template <auto F, typename... A> int unlocked(A... a) {
  Unlocked u;
  return F(a...);
}

// The call's stream, its device made current, and new memory that belongs to that stream
struct Place {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard guard;
  cudaStream_t stream;
  int dev;
  Place(PyObject *o, int d) : dev(d) {
    if (o == Py_None) {
      if (c10::cuda::current_device() != d) device.set_index(d);
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)d).stream();
      return;
    }
    PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
    PyObject *i = h ? PyObject_GetAttrString(o, "device_index") : nullptr;
    const int64_t hv = h ? PyLong_AsLongLong(h) : 0, iv = i ? PyLong_AsLongLong(i) : 0;
    Py_XDECREF(h);
    Py_XDECREF(i);
    if (PyErr_Occurred()) throw Refused();
    if (iv != d) refuse("stream: of cuda:%lld, the tensors are on cuda:%d", (long long)iv, d);
    stream = (cudaStream_t)hv;
    guard.reset_stream(c10::cuda::getStreamFromExternal(stream, (c10::DeviceIndex)d));
  }
  at::Tensor memory(at::IntArrayRef shape, at::ScalarType t) const {
    Unlocked u;
    return at::empty(shape, at::TensorOptions().dtype(t).device(at::kCUDA, (c10::DeviceIndex)dev));
  }
};

at::ScalarType type_of(int dtype) { return dtype ? at::kBFloat16 : at::kFloat; }

template <typename F> PyObject *entry(Py_ssize_t n, Py_ssize_t want, F &&f) {
  HANDLE_TH_ERRORS
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject *answer(int rc, const at::Tensor *fresh, PyObject *given) {
  if (rc) return PyLong_FromLong(rc);
  if (fresh) return THPVariable_Wrap(*fresh);
  Py_INCREF(given);
  return given;
}

// attn_packed(q, k, v, cu_seqlens, out, scale, status, stream)
PyObject *attn_packed(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return entry(n, 8, [&]() -> PyObject * {
    const at::Tensor &tq = tensor("q", a[0]), &tc = tensor("cu_seqlens", a[3]);
    if (!tq.is_cuda()) refuse("q: a CUDA tensor");
    const int dev = tq.get_device();
    const Rows q = rows("q", a[0], dev), k = rows("k", a[1], dev, ANY, q.d, q.dtype, q.n),
               v = rows("v", a[2], dev, k.h, q.d, q.dtype, q.n);
    if (q.h < 1 || k.h < 1 || q.h % k.h) refuse("%lld query heads over %lld key heads", (long long)q.h, (long long)k.h);
    if (tc.numel() < 1) refuse("cu_seqlens: int32 [prompts + 1]");
    const int32_t *cu = ints("cu_seqlens", a[3], dev, tc.numel());
    const float scale = scale_of(a[5], q.d);
    if (!(scale > 0.f)) refuse("scale: positive");
    int32_t *status = status_of(a[6], dev);
    if (q.n >= (1LL << 31) || tc.numel() > (1LL << 31)) refuse("q: below 2^31 rows and prompts");
    Place at(a[7], dev);
    at::Tensor fresh;
    Rows o;
    if (a[4] == Py_None) {
      fresh = at.memory({q.n, q.h, q.d}, type_of(q.dtype));
      o.p = fresh.data_ptr();
      o.ld = q.h * q.d;
    } else {
      o = rows("out", a[4], dev, q.h, q.d, q.dtype, q.n);
      apart("q", o, q);
      apart("k", o, k);
      apart("v", o, v);
    }
    const int rc = q.n ? unlocked<dreamer_attn_packed>(q.p, q.ld, k.p, k.ld, v.p, v.ld, o.p, o.ld, cu, (int)tc.numel() - 1,
                                             (int)q.n, (int)q.h, (int)k.h, (int)q.d, q.dtype, scale, status, at.stream)
                       : 0;
    return answer(rc, a[4] == Py_None ? &fresh : nullptr, a[4]);
  });
}

// One depth of a cache tensor uint8 [depth][batch][heads][blocks][bytes]
struct Cache {
  dreamer_kv4_cache c;
  int dev;
  int64_t depth;
  intptr_t begin, end;  // bytes of all depths
};
Cache cache_of(PyObject *data, PyObject *head_dim, PyObject *depth) {
  const at::Tensor &t = tensor("data", data);
  if (t.scalar_type() != at::kByte || t.dim() != 5 || !t.is_cuda() || !t.is_contiguous())
    refuse("data: a contiguous CUDA uint8 tensor [depth][batch][heads][blocks][bytes]");
  const int64_t d = whole(head_dim);
  if (d != 64 && d != 128) refuse("head_dim: 64 or 128");
  const int64_t block = dreamer_kv4_bytes(1, 1, (int)d, 64);
  if (t.size(4) != block || t.numel() == 0 || ((uintptr_t)t.data_ptr() & 15) || t.size(1) >= (1LL << 31) ||
      t.size(2) >= (1LL << 31) || t.size(3) >= (1LL << 25))
    refuse("data: blocks of %lld bytes, 16-byte aligned", (long long)block);
  Cache c;
  c.dev = t.get_device();
  c.depth = t.size(0);
  const int64_t l = depth ? whole(depth) : 0;
  if (l < 0 || l >= c.depth) refuse("depth: 0..%lld", (long long)c.depth - 1);
  c.begin = (intptr_t)t.data_ptr();
  c.end = c.begin + (intptr_t)t.numel();
  c.c.data = (uint8_t *)t.data_ptr() + l * t.stride(0);
  c.c.batch = (int)t.size(1);
  c.c.n_kv_heads = (int)t.size(2);
  c.c.head_dim = (int)d;
  c.c.capacity = (int)t.size(3) * 64;
  return c;
}

// Rows that the cache must not hold: outputs, and what is stored into it
void off_cache(const char *name, const Rows &x, const Cache &c) {
  if (x.n == 0) return;
  const intptr_t x0 = (intptr_t)x.p, x1 = x0 + ((x.n - 1) * x.ld + x.h * x.d) * (x.dtype ? 2 : 4);
  if (x0 < c.end && c.begin < x1) refuse("%s: overlaps the cache", name);
}

// kv4_sizes(data, head_dim) -> (depth, batch, heads, capacity)
PyObject *kv4_sizes(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return entry(n, 2, [&]() -> PyObject * {
    const Cache c = cache_of(a[0], a[1], nullptr);
    return Py_BuildValue("(Liii)", (long long)c.depth, c.c.batch, c.c.n_kv_heads, c.c.capacity);
  });
}

// kv4_store(data, head_dim, depth, k, v, cu_rows, start, status, stream)
PyObject *kv4_store(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return entry(n, 9, [&]() -> PyObject * {
    const Cache c = cache_of(a[0], a[1], a[2]);
    const Rows k = rows("k", a[3], c.dev, c.c.n_kv_heads, c.c.head_dim),
               v = rows("v", a[4], c.dev, k.h, k.d, k.dtype, k.n);
    const int32_t *cu = ints("cu_rows", a[5], c.dev, c.c.batch + 1LL), *start = ints("start", a[6], c.dev, c.c.batch);
    off_cache("k", k, c);
    off_cache("v", v, c);
    int32_t *status = status_of(a[7], c.dev);
    if (k.n >= (1LL << 31)) refuse("k: below 2^31 rows");
    Place at(a[8], c.dev);
    const int rc = k.n ? unlocked<dreamer_kv4_store>(&c.c, k.p, k.ld, v.p, v.ld, cu, start, (int)k.n, k.dtype, status, at.stream) : 0;
    return answer(rc, nullptr, Py_None);
  });
}

// kv4_load(data, head_dim, depth, cu_rows, start, n_rows, dtype (0 or 1), out_k, out_v, status, stream)
PyObject *kv4_load(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return entry(n, 11, [&]() -> PyObject * {
    const Cache c = cache_of(a[0], a[1], a[2]);
    const int64_t rows_n = whole(a[5]);
    const int dtype = (int)whole(a[6]);
    if (rows_n < 0 || rows_n >= (1LL << 31)) refuse("n_rows: not negative, below 2^31");
    const int32_t *cu = ints("cu_rows", a[3], c.dev, c.c.batch + 1LL), *start = ints("start", a[4], c.dev, c.c.batch);
    int32_t *status = status_of(a[9], c.dev);
    Place at(a[10], c.dev);
    const int64_t h = c.c.n_kv_heads, d = c.c.head_dim;
    const bool mine = a[7] == Py_None && a[8] == Py_None;  // half a pair is refused below
    at::Tensor tk, tv;
    Rows k, v;
    if (mine) {
      tk = at.memory({rows_n, h, d}, type_of(dtype));
      tv = at.memory({rows_n, h, d}, type_of(dtype));
      k.p = tk.data_ptr();
      v.p = tv.data_ptr();
      k.ld = v.ld = h * d;
    } else {
      k = rows("out[0]", a[7], c.dev, h, d, dtype, rows_n);
      v = rows("out[1]", a[8], c.dev, h, d, dtype, rows_n);
      apart("out[1]", k, v);
      off_cache("out[0]", k, c);
      off_cache("out[1]", v, c);
    }
    const int rc = rows_n ? unlocked<dreamer_kv4_load>(&c.c, k.p, k.ld, v.p, v.ld, cu, start, (int)rows_n, dtype, mine, status, at.stream) : 0;
    if (rc) return PyLong_FromLong(rc);
    return mine ? Py_BuildValue("(NN)", THPVariable_Wrap(tk), THPVariable_Wrap(tv)) : Py_BuildValue("(OO)", a[7], a[8]);
  });
}

// kv4_attend(data, head_dim, depth, q, lens, out, scale, status, stream)
PyObject *kv4_attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return entry(n, 9, [&]() -> PyObject * {
    const Cache c = cache_of(a[0], a[1], a[2]);
    const Rows q = rows("q", a[3], c.dev, ANY, c.c.head_dim, -1, c.c.batch);
    if (q.h < 1 || q.h % c.c.n_kv_heads) refuse("q: a multiple of %d heads", c.c.n_kv_heads);
    const int32_t *lens = ints("lens", a[4], c.dev, c.c.batch);
    const float scale = scale_of(a[6], q.d);
    int32_t *status = status_of(a[7], c.dev);
    Place at(a[8], c.dev);
    at::Tensor fresh, ws;
    Rows o;
    if (a[5] == Py_None) {
      fresh = at.memory({q.n, q.h, q.d}, type_of(q.dtype));
      o.p = fresh.data_ptr();
      o.ld = q.h * q.d;
    } else {
      o = rows("out", a[5], c.dev, q.h, q.d, q.dtype, q.n);
      if (o.p != q.p || o.ld != q.ld) apart("q", o, q);  // out may be q itself
      off_cache("out", o, c);
    }
    const int64_t need = dreamer_attn_kv4_workspace(&c.c, (int)q.h);
    if (need) ws = at.memory({need}, at::kByte);  // returned to the stream's pool at the end
    const int rc = unlocked<dreamer_attn_kv4>(&c.c, q.p, q.ld, o.p, o.ld, lens, (int)q.h, q.dtype, scale,
                                    need ? ws.data_ptr() : nullptr, need, status, at.stream);
    return answer(rc, a[5] == Py_None ? &fresh : nullptr, a[5]);
  });
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(attn_packed), FAST(kv4_sizes), FAST(kv4_store), FAST(kv4_load), FAST(kv4_attend), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attention", "Entry points of attention.py", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention(void) { return PyModule_Create(&module); }
