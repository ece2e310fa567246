// Calls of a decode step's latency path without ctypes: checks of the tensors and the call into
// libtg, for tg_qk_norm_rope, tg_prefill_attn and tg_prefix_attn.  Marshalling only, like the
// ctypes binding beside it; a dozen tensors checked from Python and passed through ctypes took
// 9 us a call, more than the kernels of a small step.
//
// Built as the Python module _calls.  The addresses of the libtg functions come from the ctypes
// handle (bind), so that there is one libtg and one way of loading it.
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tg.h"

#include <initializer_list>

namespace {

using Rope = decltype(&tg_qk_norm_rope);
using Prefill = decltype(&tg_prefill_attn);
using Prefix = decltype(&tg_prefix_attn);
Rope rope_fn = nullptr;
Prefill prefill_fn = nullptr;
Prefix prefix_fn = nullptr;

struct Refused {};  // a Python exception is set

const at::Tensor &tensor(PyObject *o, const char *name, int64_t dev) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA torch.Tensor", name);
    throw Refused();
  }
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) {
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA torch.Tensor", name);
    throw Refused();
  }
  if (t.get_device() != dev) {
    PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, the current device is cuda:%d", name, (int)t.get_device(), (int)dev);
    throw Refused();
  }
  return t;
}

void check_type(const at::Tensor &t, const char *name, at::ScalarType type) {
  if (t.scalar_type() == type) return;
  PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
  throw Refused();
}

void check_shape(const at::Tensor &t, const char *name, std::initializer_list<int64_t> shape) {
  if (t.sizes() == at::IntArrayRef(shape)) return;
  std::string want, got;
  for (int64_t n : shape) want += (want.empty() ? "" : ", ") + std::to_string(n);
  for (int64_t n : t.sizes()) got += (got.empty() ? "" : ", ") + std::to_string(n);
  PyErr_Format(PyExc_ValueError, "%s has shape (%s), not (%s)", name, got.c_str(), want.c_str());
  throw Refused();
}

void check_dims(const at::Tensor &t, const char *name, int64_t dims) {
  if (t.dim() == dims) return;
  PyErr_Format(PyExc_ValueError, "%s has %d dimensions, not %d", name, (int)t.dim(), (int)dims);
  throw Refused();
}

template <typename T>
T *address(const at::Tensor &t, const char *name) {
  if (!t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    throw Refused();
  }
  return static_cast<T *>(t.data_ptr());
}

// pointer of a contiguous tensor of that type on the device (and of that shape)
template <typename T>
T *arg(PyObject *o, const char *name, int64_t dev, at::ScalarType type) {
  const at::Tensor &t = tensor(o, name, dev);
  check_type(t, name, type);
  return address<T>(t, name);
}
template <typename T>
T *arg(PyObject *o, const char *name, int64_t dev, at::ScalarType type, std::initializer_list<int64_t> shape) {
  const at::Tensor &t = tensor(o, name, dev);
  check_type(t, name, type);
  check_shape(t, name, shape);
  return address<T>(t, name);
}
template <typename T, typename... Shape>
T *opt(PyObject *o, const char *name, int64_t dev, at::ScalarType type, Shape... shape) {
  return o == Py_None ? nullptr : arg<T>(o, name, dev, type, shape...);
}

int64_t integer(PyObject *o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int small(int64_t v, const char *name) {
  if (v >= INT32_MIN && v <= INT32_MAX) return (int)v;
  PyErr_Format(PyExc_ValueError, "%s=%lld leaves int32", name, (long long)v);
  throw Refused();
}
double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
void *pointer(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused();
  return p;
}
tg_stream_t stream_of(PyObject *o) { return static_cast<tg_stream_t>(pointer(o)); }

// The call itself, without the interpreter's lock, as through ctypes: a launch may wait for room in
// the stream's queue, which may wait for a host callback that needs the lock.
template <typename F, typename... A>
int unlocked(F fn, A... args) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = fn(args...);
  Py_END_ALLOW_THREADS
  return rc;
}

// no C++ exception reaches Python's C code
template <typename F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", given, wanted);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused &) {
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;

// bind(rope, prefill, prefix): addresses of the libtg functions
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 3, [&] {
    rope_fn = reinterpret_cast<Rope>(pointer(a[0]));
    prefill_fn = reinterpret_cast<Prefill>(pointer(a[1]));
    prefix_fn = reinterpret_cast<Prefix>(pointer(a[2]));
    return 0;
  });
}

// (stream, device, qkv, cu_q, start, cos_sin, q, K, V, q_weight, k_weight, eps, pairs, positions, dev_status)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const int64_t dev = integer(a[1]);
    const at::Tensor &q = tensor(a[6], "q", dev), &K = tensor(a[7], "K", dev), &qkv = tensor(a[2], "qkv", dev);
    check_dims(q, "q", 3), check_dims(K, "K", 4);
    const int64_t T = q.size(0), H_q = q.size(1), d = q.size(2), batch = K.size(0), H = K.size(1), Nmax = K.size(2);
    const int64_t heads = H_q + 2 * H;
    check_type(qkv, "qkv", kBf16), check_type(q, "q", kBf16), check_type(K, "K", kBf16);
    check_shape(qkv, "qkv", {T, heads, d}), check_shape(K, "K", {batch, H, Nmax, d});
    if (T && (qkv.stride(2) != 1 || qkv.stride(1) != d)) {
      PyErr_SetString(PyExc_ValueError, "qkv must have contiguous token rows");
      throw Refused();
    }
    int64_t max_pos = 0, rot = 0;
    const float *table = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor &t = tensor(a[5], "cos_sin", dev);
      check_dims(t, "cos_sin", 3);
      max_pos = t.size(0), rot = 2 * t.size(1);
      table = arg<float>(a[5], "cos_sin", dev, kF32, {max_pos, t.size(1), 2});
    }
    const int yes = PyObject_IsTrue(a[12]);
    if (yes < 0) throw Refused();
    return unlocked(
        rope_fn, stream_of(a[0]), small(batch, "batch"), small(T, "T"), small(H_q, "H_q"), small(H, "H"), small(d, "d"),
        small(Nmax, "Nmax"), small(rot, "rot"), small(max_pos, "max_pos"), yes ? TG_ROPE_PAIRS : 0u,
        arg<int32_t>(a[3], "cu_q", dev, kI32, {batch + 1}), arg<int32_t>(a[4], "start", dev, kI32, {batch}),
        static_cast<uint16_t *>(qkv.data_ptr()), T > 1 ? qkv.stride(0) : heads * d,
        opt<float>(a[9], "q_weight", dev, kF32, std::initializer_list<int64_t>{d}),
        opt<float>(a[10], "k_weight", dev, kF32, std::initializer_list<int64_t>{d}), (float)real(a[11]),
        opt<int32_t>(a[13], "positions", dev, kI32, std::initializer_list<int64_t>{T}), table, address<uint16_t>(q, "q"),
        address<uint16_t>(K, "K"), arg<uint16_t>(a[8], "V", dev, kBf16, {batch, H, Nmax, d}),
        opt<int32_t>(a[14], "dev_status", dev, kI32));
  });
}

struct Workspace {
  void *at = nullptr;
  int64_t bytes = 0;
  Workspace(PyObject *o, int64_t dev) {
    if (o == Py_None) return;
    at = arg<uint8_t>(o, "workspace", dev, at::kByte);
    bytes = THPVariable_Unpack(o).numel();
  }
};

// (stream, device, plan host, plan device, q, K, V, scale, out, lse, workspace, dev_status)
PyObject *prefill_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const int64_t dev = integer(a[1]);
    const tg_tile_header *hd = static_cast<const tg_tile_header *>(pointer(a[2]));
    const at::Tensor &K = tensor(a[5], "K", dev);
    check_dims(K, "K", 4);
    const int64_t Nmax = K.size(2);
    const Workspace ws(a[10], dev);
    return unlocked(prefill_fn, stream_of(a[0]), hd, pointer(a[3]),
                    arg<uint16_t>(a[4], "q", dev, kBf16, {hd->rows, hd->H_q, hd->d}),
                    arg<uint16_t>(a[5], "K", dev, kBf16, {hd->batch, hd->H, Nmax, hd->d}),
                    arg<uint16_t>(a[6], "V", dev, kBf16, {hd->batch, hd->H, Nmax, hd->d}), small(Nmax, "Nmax"),
                    (float)real(a[7]), ws.at, ws.bytes,
                    arg<uint16_t>(a[8], "out", dev, kBf16, {hd->rows, hd->H_q, hd->d}),
                    opt<float>(a[9], "lse", dev, kF32, std::initializer_list<int64_t>{hd->rows, hd->H_q}),
                    opt<int32_t>(a[11], "dev_status", dev, kI32));
  });
}

// (stream, device, plan host, plan device, q, pool, pool_pages, pt_off, pt_ids, scale, own_out, own_lse, out,
//  lse, workspace, dev_status)
PyObject *prefix_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    const int64_t dev = integer(a[1]), pages = integer(a[6]);
    const tg_tile_header *hd = static_cast<const tg_tile_header *>(pointer(a[2]));
    const at::Tensor &pool = tensor(a[5], "pool", dev);
    check_type(pool, "pool", kBf16);
    const int64_t page = (int64_t)hd->H_p * 2 * hd->P * hd->d, held = page ? pool.numel() / page : 0;
    if (pages > held) {
      PyErr_Format(PyExc_ValueError, "pool holds %lld pages, not %lld", (long long)held, (long long)pages);
      throw Refused();
    }
    const int64_t lists = (int64_t)hd->groups * (hd->H_p ? hd->H / hd->H_p : 0);
    const Workspace ws(a[14], dev);
    return unlocked(
        prefix_fn, stream_of(a[0]), hd, pointer(a[3]), arg<uint16_t>(a[4], "q", dev, kBf16, {hd->rows, hd->H_q, hd->d}),
        address<uint16_t>(pool, "pool"), pages, arg<int64_t>(a[7], "pt_off", dev, at::kLong, {lists + 1}),
        arg<int32_t>(a[8], "pt_ids", dev, kI32), (float)real(a[9]),
        opt<uint16_t>(a[10], "own_out", dev, kBf16, std::initializer_list<int64_t>{hd->rows, hd->H_q, hd->d}),
        opt<float>(a[11], "own_lse", dev, kF32, std::initializer_list<int64_t>{hd->rows, hd->H_q}), ws.at, ws.bytes,
        arg<uint16_t>(a[12], "out", dev, kBf16, {hd->rows, hd->H_q, hd->d}),
        opt<float>(a[13], "lse", dev, kF32, std::initializer_list<int64_t>{hd->rows, hd->H_q}),
        opt<int32_t>(a[15], "dev_status", dev, kI32));
  });
}

PyMethodDef methods[] = {{"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
                         {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)),
                          METH_FASTCALL, nullptr},
                         {"prefill_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefill_attn)),
                          METH_FASTCALL, nullptr},
                         {"prefix_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_attn)),
                          METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
