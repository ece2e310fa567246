// Calls of a decode step's latency path without ctypes: checks of the tensors and the call into
// libtg, for tg_qk_norm_rope, tg_prefill_attn and tg_prefix_attn, and for tg_append_rope,
// tg_decode_grown, tg_quant_pages and tg_dequant_pages.  Marshalling only, like the
// ctypes binding beside it; a dozen tensors checked from Python and passed through ctypes took
// 9 us a call, more than the kernels of a small step.
//
// Built as the Python module _calls.  The addresses of the libtg functions come from the ctypes
// handle (bind, bind_pages), so that there is one libtg and one way of loading it.
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
using Append = decltype(&tg_append_rope);
using Grown = decltype(&tg_decode_grown);
using Quant = decltype(&tg_quant_pages);
using Dequant = decltype(&tg_dequant_pages);
Append append_fn = nullptr;
Grown grown_fn = nullptr;
Quant quant_fn = nullptr;
Dequant dequant_fn = nullptr;

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

// bind_pages(append, grown, quant, dequant): addresses of the libtg functions
PyObject *bind_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    append_fn = reinterpret_cast<Append>(pointer(a[0]));
    grown_fn = reinterpret_cast<Grown>(pointer(a[1]));
    quant_fn = reinterpret_cast<Quant>(pointer(a[2]));
    dequant_fn = reinterpret_cast<Dequant>(pointer(a[3]));
    return 0;
  });
}

// A pool of `pages` pages of the format: bf16, or bytes for 4-bit pages.
void *pool_arg(PyObject *o, int64_t dev, int format, int64_t pages, int64_t H_p, int64_t P, int64_t d,
               const char *name = "pool") {
  const at::Tensor &pool = tensor(o, name, dev);
  const bool bf16 = format == TG_PAGES_BF16;
  check_type(pool, name, bf16 ? kBf16 : at::kByte);
  const int64_t page = bf16 ? H_p * 2 * P * d : H_p * (P / 16) * (d / 128) * TG_TILE4_BYTES;
  const int64_t held = page > 0 ? pool.numel() / page : 0;
  if (pages > held) {
    PyErr_Format(PyExc_ValueError, "%s holds %lld pages, not %lld", name, (long long)held, (long long)pages);
    throw Refused();
  }
  return address<void>(pool, name);
}

// (stream, device, qkv, cu_q, cos_sin, q, pool, pool_pages, head_order, ntok, added, reserve, pt_off, pt_ids, H_p, P,
//  format, k_unit, v_unit, q_weight, k_weight, eps, pairs, positions, axis_of (bytes), origin, K, V, start, dev_status)
PyObject *append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 30, [&] {
    const int64_t dev = integer(a[1]);
    const at::Tensor &qkv = tensor(a[2], "qkv", dev), &q = tensor(a[5], "q", dev), &ntok = tensor(a[9], "ntok", dev);
    check_dims(q, "q", 3), check_dims(ntok, "ntok", 2);
    const int64_t T = q.size(0), H_q = q.size(1), d = q.size(2), batch = ntok.size(0), H = ntok.size(1);
    const int64_t heads = H_q + 2 * H, pages = integer(a[7]);
    const int H_p = small(integer(a[14]), "H_p"), P = small(integer(a[15]), "P"), format = small(integer(a[16]), "format");
    const int64_t lists = H_p > 0 ? batch * (H / H_p) : 0;
    check_type(qkv, "qkv", kBf16), check_type(q, "q", kBf16);
    check_shape(qkv, "qkv", {T, heads, d});
    if (T && (qkv.stride(2) != 1 || qkv.stride(1) != d)) {
      PyErr_SetString(PyExc_ValueError, "qkv must have contiguous token rows");
      throw Refused();
    }
    int64_t max_pos = 0, rot = 0, axes = 1;
    const float *table = nullptr;
    if (a[4] != Py_None) {
      const at::Tensor &t = tensor(a[4], "cos_sin", dev);
      check_dims(t, "cos_sin", 3);
      max_pos = t.size(0), rot = 2 * t.size(1);
      table = arg<float>(a[4], "cos_sin", dev, kF32, {max_pos, t.size(1), 2});
    }
    const int32_t *positions = nullptr;
    if (a[23] != Py_None) {
      const at::Tensor &t = tensor(a[23], "positions", dev);
      if (t.dim() == 2) axes = t.size(1);
      positions = t.dim() == 2 ? arg<int32_t>(a[23], "positions", dev, kI32, {T, axes})
                               : arg<int32_t>(a[23], "positions", dev, kI32, {T});
    }
    const uint8_t *axis_of = nullptr;
    if (a[24] != Py_None) {
      if (!PyBytes_Check(a[24]) || PyBytes_GET_SIZE(a[24]) != rot / 2) {
        PyErr_Format(PyExc_ValueError, "axis_of must have an axis for each of the %lld pairs", (long long)(rot / 2));
        throw Refused();
      }
      axis_of = reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(a[24]));
    }
    int64_t Nmax = 0;
    uint16_t *K = nullptr, *V = nullptr;
    if (a[26] != Py_None) {
      const at::Tensor &t = tensor(a[26], "K", dev);
      check_dims(t, "K", 4);
      Nmax = t.size(2);
      K = arg<uint16_t>(a[26], "K", dev, kBf16, {batch, H, Nmax, d});
    }
    if (a[27] != Py_None) V = arg<uint16_t>(a[27], "V", dev, kBf16, {batch, H, Nmax, d});
    const int yes = PyObject_IsTrue(a[22]);
    if (yes < 0) throw Refused();
    return unlocked(
        append_fn, stream_of(a[0]), small(batch, "batch"), small(T, "T"), small(H_q, "H_q"), small(H, "H"), H_p, P,
        small(d, "d"), small(rot, "rot"), small(max_pos, "max_pos"), yes ? TG_ROPE_PAIRS : 0u,
        arg<int32_t>(a[3], "cu_q", dev, kI32, {batch + 1}), static_cast<const uint16_t *>(qkv.data_ptr()),
        T > 1 ? qkv.stride(0) : heads * d, opt<float>(a[19], "q_weight", dev, kF32, std::initializer_list<int64_t>{d}),
        opt<float>(a[20], "k_weight", dev, kF32, std::initializer_list<int64_t>{d}), (float)real(a[21]),
        small(axes, "axes"), positions, axis_of,
        opt<int32_t>(a[25], "origin", dev, kI32, std::initializer_list<int64_t>{batch}), table,
        arg<int32_t>(a[8], "head_order", dev, kI32, {H}), arg<int32_t>(a[9], "ntok", dev, kI32),
        opt<int32_t>(a[10], "added", dev, kI32, std::initializer_list<int64_t>{batch}), small(integer(a[11]), "reserve"),
        arg<int64_t>(a[12], "pt_off", dev, at::kLong, {lists + 1}), arg<int32_t>(a[13], "pt_ids", dev, kI32), format,
        (float)real(a[17]), (float)real(a[18]), pool_arg(a[6], dev, format, pages, H_p, P, d), pages,
        address<uint16_t>(q, "q"), K, V, small(Nmax, "Nmax"),
        opt<int32_t>(a[28], "start", dev, kI32, std::initializer_list<int64_t>{batch}),
        opt<int32_t>(a[29], "dev_status", dev, kI32));
  });
}

// (stream, device, to 4 bits, head_order, ntok, added, plus, reserve, H_p, P, d, src_off, src_ids, src, src_pages, dst_off,
//  dst_ids, dst, dst_pages, k_unit, v_unit, dev_status)
PyObject *convert_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 22, [&] {
    const int64_t dev = integer(a[1]), src_pages = integer(a[14]), dst_pages = integer(a[18]);
    const bool to4 = PyObject_IsTrue(a[2]) == 1;
    const at::Tensor &ntok = tensor(a[4], "ntok", dev);
    check_dims(ntok, "ntok", 2);
    const int batch = small(ntok.size(0), "batch"), H = small(ntok.size(1), "H");
    const int H_p = small(integer(a[8]), "H_p"), P = small(integer(a[9]), "P"), d = small(integer(a[10]), "d");
    const int64_t lists = H_p > 0 ? (int64_t)batch * (H / H_p) : 0;
    const tg_stream_t stream = stream_of(a[0]);
    const int32_t *order = arg<int32_t>(a[3], "head_order", dev, kI32, {H}), *counts = arg<int32_t>(a[4], "ntok", dev, kI32);
    const int32_t *added = opt<int32_t>(a[5], "added", dev, kI32, std::initializer_list<int64_t>{batch});
    const int plus = small(integer(a[6]), "plus"), reserve = small(integer(a[7]), "reserve");
    const int64_t *src_off = arg<int64_t>(a[11], "src_off", dev, at::kLong, {lists + 1});
    const int64_t *dst_off = arg<int64_t>(a[15], "dst_off", dev, at::kLong, {lists + 1});
    const int32_t *src_ids = arg<int32_t>(a[12], "src_ids", dev, kI32), *dst_ids = arg<int32_t>(a[16], "dst_ids", dev, kI32);
    void *src = pool_arg(a[13], dev, to4 ? TG_PAGES_BF16 : TG_PAGES_E2M1, src_pages, H_p, P, d, "src");
    void *dst = pool_arg(a[17], dev, to4 ? TG_PAGES_E2M1 : TG_PAGES_BF16, dst_pages, H_p, P, d, "dst");
    const float k_unit = (float)real(a[19]), v_unit = (float)real(a[20]);
    int32_t *status = opt<int32_t>(a[21], "dev_status", dev, kI32);
    if (to4)
      return unlocked(quant_fn, stream, batch, H, H_p, P, d, order, counts, src_off, src_ids,
                      static_cast<const uint16_t *>(src), src_pages, dst_off, dst_ids, dst, dst_pages, k_unit, v_unit, status);
    return unlocked(dequant_fn, stream, batch, H, H_p, P, d, order, counts, added, plus, reserve, src_off, src_ids,
                    static_cast<const void *>(src), src_pages, dst_off, dst_ids, static_cast<uint16_t *>(dst), dst_pages, k_unit,
                    v_unit, status);
  });
}

// (stream, device, plan host, plan device, layer, format, q, pool, pool_pages, pt_off, pt_ids, ntok, added, plus, reserve,
//  scale, k_unit, v_unit, out, lse, workspace, dev_status, cta_time)
PyObject *decode_grown(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 23, [&] {
    const int64_t dev = integer(a[1]), pages = integer(a[8]);
    const tg_plan_header *hd = static_cast<const tg_plan_header *>(pointer(a[2]));
    const int format = small(integer(a[5]), "format");
    const int64_t lists = (int64_t)hd->batch * hd->G;
    const Workspace ws(a[20], dev);
    return unlocked(
        grown_fn, stream_of(a[0]), hd, pointer(a[3]), small(integer(a[4]), "layer"), format,
        arg<uint16_t>(a[6], "q", dev, kBf16, {hd->batch, hd->H_q, hd->d}),
        pool_arg(a[7], dev, format, pages, hd->H_p, hd->P, hd->d), pages,
        arg<int64_t>(a[9], "pt_off", dev, at::kLong, {lists + 1}), arg<int32_t>(a[10], "pt_ids", dev, kI32),
        arg<int32_t>(a[11], "ntok", dev, kI32, {hd->batch, hd->H}),
        opt<int32_t>(a[12], "added", dev, kI32, std::initializer_list<int64_t>{hd->batch}), small(integer(a[13]), "plus"),
        small(integer(a[14]), "reserve"), (float)real(a[15]), (float)real(a[16]), (float)real(a[17]), ws.at, ws.bytes,
        arg<uint16_t>(a[18], "out", dev, kBf16, {hd->batch, hd->H_q, hd->d}),
        opt<float>(a[19], "lse", dev, kF32, std::initializer_list<int64_t>{hd->batch, hd->H_q}),
        opt<int32_t>(a[21], "dev_status", dev, kI32),
        opt<int64_t>(a[22], "cta_time", dev, at::kLong, std::initializer_list<int64_t>{2 * (int64_t)hd->N_CTA}));
  });
}

PyMethodDef methods[] = {{"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
                         {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)),
                          METH_FASTCALL, nullptr},
                         {"prefill_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefill_attn)),
                          METH_FASTCALL, nullptr},
                         {"prefix_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_attn)),
                          METH_FASTCALL, nullptr},
                         {"bind_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_pages)),
                          METH_FASTCALL, nullptr},
                         {"append_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_rope)),
                          METH_FASTCALL, nullptr},
                         {"convert_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(convert_pages)),
                          METH_FASTCALL, nullptr},
                         {"decode_grown", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_grown)),
                          METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
