// CPython binding of the token-by-token entry points (dl.h, c1-c4).
//
// These calls run for a few microseconds, so their marshalling counts: read
// attribute by attribute in Python, a call of fourteen buffers took 7 us before
// it reached the library; here it takes under one.  Tensors are viewed through
// the C exchange table that torch.Tensor carries for this purpose (DLPack's
// DLPackExchangeAPI), so nothing here depends on torch's C++ interface; the
// library is called through the addresses that bind() is given.
//
// Every buffer must be a contiguous tensor of the stated type and number of
// elements on the current CUDA device (the call launches there); a mismatch is
// a ValueError, before the library is called.  Returns the dl_status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>

#include <cstring>
#include <initializer_list>

#include "dl.h"

namespace {

const DLPackExchangeAPI* g_api = nullptr;
PyTypeObject* g_tensor = nullptr;
PyObject* g_current_device = nullptr;  // callable: index of the current CUDA device

decltype(&dl_qk_norm_rope) g_rope = nullptr;
decltype(&dl_decode_attn) g_decode = nullptr;
decltype(&dl_evict_select) g_evict = nullptr;
decltype(&dl_cache_compact) g_compact = nullptr;

// A number of elements; more than 64 bits hold is more than any tensor has.
int64_t product(std::initializer_list<int64_t> v) {
  int64_t p = 1;
  for (int64_t x : v)
    if (__builtin_mul_overflow(p, x, &p)) return INT64_MAX;
  return p;
}

// A call in the making.  The first failure sets the Python error and stays.
struct Call {
  const char* name;
  PyObject* const* args;
  dl_attn_desc desc;
  int dev = -1;
  bool ok = true;

  Call(const char* name_, PyObject* const* args_, Py_ssize_t nargs, Py_ssize_t want)
      : name(name_), args(args_) {
    if (!g_rope) {
      fail(PyExc_RuntimeError, "not bound: this torch has no DLPack exchange table on torch.Tensor");
    } else if (nargs != want) {
      fail(PyExc_TypeError, "wrong number of arguments");
    } else {
      Py_buffer view;
      if (PyObject_GetBuffer(args[0], &view, PyBUF_SIMPLE) != 0) {
        ok = false;
        return;
      }
      const bool size = view.len == (Py_ssize_t)sizeof(desc);
      if (size) std::memcpy(&desc, view.buf, sizeof(desc));
      PyBuffer_Release(&view);
      if (!size) fail(PyExc_TypeError, "desc is not a dl_attn_desc");
    }
  }

  void fail(PyObject* type, const char* what) {
    if (ok) PyErr_Format(type, "%s: %s", name, what);
    ok = false;
  }

  int dtype_code() const { return desc.dtype == DL_BF16 ? kDLBfloat : kDLFloat; }
  int dtype_bits() const { return desc.dtype == DL_BF16 ? 16 : 32; }

  bool view(PyObject* o, const char* what, DLTensor* t) {
    if (!ok) return false;
    if (!PyObject_TypeCheck(o, g_tensor)) {
      PyErr_Format(PyExc_TypeError, "%s: %s must be a torch.Tensor, got %s", name, what, Py_TYPE(o)->tp_name);
      return ok = false;
    }
    if (g_api->dltensor_from_py_object_no_sync(o, t) != 0) return ok = false;
    if (dev < 0 && t->device.device_type == kDLCUDA) {
      PyObject* d = PyObject_CallNoArgs(g_current_device);
      if (!d) return ok = false;
      dev = (int)PyLong_AsLong(d);
      Py_DECREF(d);
    }
    return true;
  }

  void refuse(PyObject* o, const char* what, const char* must) {
    if (!ok) return;
    ok = false;
    PyObject* said[3];
    const char* names[3] = {"shape", "dtype", "device"};
    for (int i = 0; i < 3; ++i) {
      said[i] = PyObject_GetAttrString(o, names[i]);
      if (!said[i]) { PyErr_Clear(); said[i] = PyUnicode_FromString("?"); }
    }
    PyErr_Format(PyExc_ValueError, "%s: %s must be %s on the current CUDA device, got a tensor of shape %S and "
                 "type %S on %S", name, what, must, said[0], said[1], said[2]);
    for (PyObject* x : said) Py_XDECREF(x);
  }

  static bool contiguous(const DLTensor& t) {
    int64_t step = 1;
    bool plain = true;
    for (int i = t.ndim - 1; i >= 0; --i) {
      if (t.shape[i] == 0) return true;  // no elements at all
      if (t.shape[i] != 1 && t.strides && t.strides[i] != step) plain = false;
      step *= t.shape[i];
    }
    return plain;
  }

  static void* pointer(const DLTensor& t) { return static_cast<char*>(t.data) + t.byte_offset; }

  // Data pointer of argument i: n elements (-1: any number) of the type; None
  // and tensors without elements give NULL.
  void* buf(int i, const char* what, int code, int bits, int64_t n, int64_t* elements = nullptr) {
    PyObject* o = args[i];
    if (!ok || o == Py_None) return nullptr;
    DLTensor t;
    if (!view(o, what, &t)) return nullptr;
    int64_t have = 1;
    for (int k = 0; k < t.ndim; ++k) have *= t.shape[k];
    const bool type = code < 0 || (t.dtype.code == code && t.dtype.bits == bits && t.dtype.lanes == 1);
    if (!type || (n >= 0 && have != n) || t.device.device_type != kDLCUDA || t.device.device_id != dev ||
        !contiguous(t)) {
      char must[96];
      const char* kind = code == kDLBfloat ? "bfloat16" : code == kDLInt ? "int32" : code == kDLFloat ? "float32" : "any";
      if (n >= 0) PyOS_snprintf(must, sizeof(must), "a contiguous %s tensor of %lld elements", kind, (long long)n);
      else PyOS_snprintf(must, sizeof(must), "a contiguous %s tensor", kind);
      refuse(o, what, must);
      return nullptr;
    }
    if (elements) *elements = have * ((t.dtype.bits + 7) / 8);
    return have ? pointer(t) : nullptr;
  }
  void* data(int i, const char* what, int64_t n) { return buf(i, what, dtype_code(), dtype_bits(), n); }
  int32_t* i32(int i, const char* what, int64_t n) { return static_cast<int32_t*>(buf(i, what, kDLInt, 32, n)); }
  float* f32(int i, const char* what, int64_t n) { return static_cast<float*>(buf(i, what, kDLFloat, 32, n)); }

  // Sizes of a 3-dimensional argument [batch][rows][columns]; false: None.
  bool rows_of(int i, const char* what, int64_t* rows, int64_t* columns) {
    if (!ok || args[i] == Py_None) return false;
    DLTensor t;
    if (!view(args[i], what, &t)) return false;
    if (t.ndim != 3 || t.shape[1] > INT32_MAX || t.shape[2] > INT32_MAX) {
      refuse(args[i], what, "a [batch][n_mass][...] tensor");
      return false;
    }
    *rows = t.shape[1];
    if (columns) *columns = t.shape[2];
    return true;
  }

  int integer(int i, const char* what) {
    if (!ok) return 0;
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(args[i], &over);
    if (v == -1 && !over && PyErr_Occurred()) { ok = false; return 0; }
    if (over || v < INT32_MIN || v > INT32_MAX) {
      PyErr_Format(PyExc_ValueError, "%s: %s does not fit 32 bits", name, what);
      ok = false;
    }
    return (int)v;
  }
  float real(int i) {
    if (!ok) return 0.0f;
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return (float)v;
  }
  // None: the current stream of the device; else a raw handle.
  void* stream(int i) {
    if (!ok) return nullptr;
    void* s = nullptr;
    if (args[i] == Py_None) {
      if (dev >= 0 && g_api->current_work_stream(kDLCUDA, dev, &s) != 0) ok = false;
    } else {
      s = PyLong_AsVoidPtr(args[i]);
      if (!s && PyErr_Occurred()) ok = false;
    }
    return s;
  }
};

template <typename F>
PyObject* run(Call& c, F f) {
  if (!c.ok) return nullptr;
  if (c.dev < 0) {
    PyErr_Format(PyExc_ValueError, "%s: buffers must be on the current CUDA device", c.name);
    return nullptr;
  }
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// desc, qkv, pos, q_weight, k_weight, eps, inv_freq, Q_out, K_out, V_out, start,
// page_table, K_pool, V_pool, end, tok_pos, tok_mass, interleaved, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  Call c("dl_qk_norm_rope", args, nargs, 19);
  if (!c.ok) return nullptr;
  const int64_t B = c.desc.batch, H = c.desc.H, H_kv = c.desc.H_kv, d = c.desc.d;
  DLTensor x;
  if (!c.view(args[1], "qkv", &x)) return nullptr;
  const int64_t width = product({H + 2 * H_kv, d});
  int64_t n = 0, stride = 0;
  bool fits = x.ndim == 3 && x.dtype.code == c.dtype_code() && x.dtype.bits == c.dtype_bits() &&
              x.device.device_type == kDLCUDA && x.device.device_id == c.dev && x.shape[0] == B &&
              x.shape[1] >= 1 && x.shape[1] <= INT32_MAX && x.shape[2] >= width && x.strides &&
              x.strides[2] == 1;
  if (fits) {
    n = x.shape[1];
    // equal steps between all tokens; the strides of single ones say nothing, and a token alone has none
    stride = n > 1 ? x.strides[1] : B > 1 ? x.strides[0] : width;
    fits = (stride >= x.shape[2] || (n == 1 && B == 1)) && (B == 1 || n == 1 || x.strides[0] == n * stride);
  }
  if (!fits) {
    char must[160];
    PyOS_snprintf(must, sizeof(must), "[%lld][n_tok][>= (H + 2 H_kv) d = %lld] of the descriptor's type, with unit "
                  "stride and equal steps between tokens,", (long long)B, (long long)width);
    c.refuse(args[1], "qkv", must);
    return nullptr;
  }
  const int64_t pool = product({c.desc.n_slots, H_kv, c.desc.page, d});
  int64_t n_mass = 1, freq = 0;
  if (!c.rows_of(15, "tok_pos", &n_mass, nullptr)) c.rows_of(16, "tok_mass", &n_mass, nullptr);
  const int64_t book = product({B, n_mass, c.desc.L_ctx});
  int32_t* pos = c.i32(2, "pos", product({B, n}));
  void *qw = c.data(3, "q_weight", d), *kw = c.data(4, "k_weight", d);
  const float eps = c.real(5);
  float* f = static_cast<float*>(c.buf(6, "inv_freq", kDLFloat, 32, -1, &freq));
  void *q = c.data(7, "Q_out", product({B, H, n, d}));
  void *k = c.data(8, "K_out", product({B, H_kv, n, d})), *v = c.data(9, "V_out", product({B, H_kv, n, d}));
  int32_t *start = c.i32(10, "start", B), *table = c.i32(11, "page_table", product({B, c.desc.n_pages}));
  void *kp = c.data(12, "K_pool", pool), *vp = c.data(13, "V_pool", pool);
  int32_t *end = c.i32(14, "end", B), *tp = c.i32(15, "tok_pos", book);
  float* tm = c.f32(16, "tok_mass", book);
  const int inter = c.integer(17, "interleaved");
  void* st = c.stream(18);
  if (c.ok && freq / 4 > d) c.fail(PyExc_ValueError, "inv_freq has more than d / 2 elements");
  return run(c, [&] {
    return g_rope(&c.desc, Call::pointer(x), stride, (int)n, pos, qw, kw, eps, f, (int)(freq / 2), inter, q, k, v,
                  start, table, kp, vp, end, tp, tm, (int)n_mass, st);
  });
}

// desc, Q, K_pool, V_pool, page_table, ctx_len, O, lse, ws, tok_mass, decay, stream
PyObject* decode_attn(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  Call c("dl_decode_attn", args, nargs, 12);
  if (!c.ok) return nullptr;
  const int64_t B = c.desc.batch, H = c.desc.H, d = c.desc.d,
                pool = product({c.desc.n_slots, c.desc.H_kv, c.desc.page, d});
  int64_t n_mass = 1, ws_bytes = 0;
  c.rows_of(9, "tok_mass", &n_mass, nullptr);
  void* q = c.data(1, "Q", product({B, H, d}));
  void *kp = c.data(2, "K_pool", pool), *vp = c.data(3, "V_pool", pool);
  int32_t *table = c.i32(4, "page_table", product({B, c.desc.n_pages})), *len = c.i32(5, "ctx_len", B);
  void* o = c.data(6, "O", product({B, H, d}));
  float* lse = c.f32(7, "lse", product({B, H}));
  void* ws = c.buf(8, "ws", -1, 0, -1, &ws_bytes);
  float* mass = c.f32(9, "tok_mass", product({B, n_mass, c.desc.L_ctx}));
  const float decay = c.real(10);
  void* st = c.stream(11);
  return run(c, [&] {
    return g_decode(&c.desc, q, kp, vp, table, len, o, lse, mass, (int)n_mass, decay, ws, (size_t)ws_bytes, st);
  });
}

// desc, tok_mass, tok_pos, ctx_len, budget, n_first, n_recent, hole_idx,
// fill_idx, move_cnt, new_len, stream
PyObject* evict_select(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  Call c("dl_evict_select", args, nargs, 12);
  if (!c.ok) return nullptr;
  const int64_t B = c.desc.batch;
  int64_t n_mass = 1, rows = 0, max_move = 0;
  c.rows_of(1, "tok_mass", &n_mass, nullptr);
  c.rows_of(7, "hole_idx", &rows, &max_move);
  const int64_t book = product({B, n_mass, c.desc.L_ctx}), moves = product({B, n_mass, max_move});
  float* mass = c.f32(1, "tok_mass", book);
  int32_t *pos = c.i32(2, "tok_pos", book), *len = c.i32(3, "ctx_len", B);
  const int budget = c.integer(4, "budget"), n_first = c.integer(5, "n_first"), n_recent = c.integer(6, "n_recent");
  int32_t *hole = c.i32(7, "hole_idx", moves), *fill = c.i32(8, "fill_idx", moves);
  int32_t *cnt = c.i32(9, "move_cnt", product({B, n_mass})), *now = c.i32(10, "new_len", B);
  void* st = c.stream(11);
  return run(c, [&] {
    return g_evict(&c.desc, mass, pos, (int)n_mass, len, budget, n_first, n_recent, hole, fill, (int)max_move, cnt,
                   now, st);
  });
}

// desc, hole_idx, fill_idx, move_cnt, page_table, K_pool, V_pool, tok_pos,
// tok_mass, stream
PyObject* cache_compact(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  Call c("dl_cache_compact", args, nargs, 10);
  if (!c.ok) return nullptr;
  const int64_t B = c.desc.batch, pool = product({c.desc.n_slots, c.desc.H_kv, c.desc.page, c.desc.d});
  int64_t n_mass = 1, max_move = 0;
  c.rows_of(1, "hole_idx", &n_mass, &max_move);
  const int64_t book = product({B, n_mass, c.desc.L_ctx}), moves = product({B, n_mass, max_move});
  int32_t *hole = c.i32(1, "hole_idx", moves), *fill = c.i32(2, "fill_idx", moves);
  int32_t *cnt = c.i32(3, "move_cnt", product({B, n_mass})), *table = c.i32(4, "page_table", product({B, c.desc.n_pages}));
  void *kp = c.data(5, "K_pool", pool), *vp = c.data(6, "V_pool", pool);
  int32_t* tp = c.i32(7, "tok_pos", book);
  float* tm = c.f32(8, "tok_mass", book);
  void* st = c.stream(9);
  return run(c, [&] {
    return g_compact(&c.desc, hole, fill, cnt, (int)max_move, (int)n_mass, table, kp, vp, tp, tm, st);
  });
}

// tensor type, current-device callable, addresses of the four entry points
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *type, *device, *p[4];
  if (!PyArg_ParseTuple(args, "OOOOOO", &type, &device, &p[0], &p[1], &p[2], &p[3])) return nullptr;
  PyObject* capsule = PyObject_GetAttrString(type, "__dlpack_c_exchange_api__");
  if (!capsule) return nullptr;
  auto* api = static_cast<const DLPackExchangeAPI*>(PyCapsule_GetPointer(capsule, "dlpack_exchange_api"));
  Py_DECREF(capsule);
  if (!api) return nullptr;
  if (api->header.version.major != DLPACK_MAJOR_VERSION)
    return PyErr_Format(PyExc_ImportError, "torch's DLPack exchange table is version %u, built for %u",
                        api->header.version.major, (unsigned)DLPACK_MAJOR_VERSION);
  void* f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(p[i]);
    if (!f[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "NULL entry point");
  }
  Py_INCREF(type);
  Py_INCREF(device);
  g_tensor = reinterpret_cast<PyTypeObject*>(type);
  g_current_device = device;
  g_api = api;
  std::memcpy(&g_rope, &f[0], sizeof(void*));
  std::memcpy(&g_decode, &f[1], sizeof(void*));
  std::memcpy(&g_evict, &f[2], sizeof(void*));
  std::memcpy(&g_compact, &f[3], sizeof(void*));
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", bind, METH_VARARGS, "Sets the tensor type, the current-device callable and the entry points."},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"decode_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode_attn)), METH_FASTCALL, nullptr},
    {"evict_select", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(evict_select)), METH_FASTCALL, nullptr},
    {"cache_compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_compact)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", "Marshalling of the token-by-token calls.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  // object layouts differ between minor versions, and nothing in the file's name says which it was built for
  char built[16];
  const int n = PyOS_snprintf(built, sizeof(built), "%d.%d.", PY_MAJOR_VERSION, PY_MINOR_VERSION);
  if (std::strncmp(Py_GetVersion(), built, n) != 0)
    return PyErr_Format(PyExc_ImportError, "built for Python %d.%d, this is %s", PY_MAJOR_VERSION, PY_MINOR_VERSION,
                        Py_GetVersion());
  return PyModule_Create(&g_module);
}
