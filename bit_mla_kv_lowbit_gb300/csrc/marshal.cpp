// The Python binding's way to the serving-step calls.
//
// These calls' kernels take a few microseconds each, and so does asking a dozen
// tensors for type, device, layout, shape and address through Python attributes
// and converting twenty arguments for a foreign call.  Here a call's arguments
// are checked and it is launched in one pass: a launch and about half a
// microsecond.  A function returns the library's status, or None when an argument
// is not as it should be or the tensors are not on the current device: the
// binding then goes through them in Python, which names the fault.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mla_lowbit.h"

namespace {

struct Library {
  decltype(&mla_lowbit_page_bytes) page_bytes;
  decltype(&mla_lowbit_assign) assign;
  decltype(&mla_lowbit_norm_rope) norm_rope;
  decltype(&mla_lowbit_norm_rope_write) norm_rope_write;
  decltype(&mla_lowbit_read) read;
  decltype(&mla_lowbit_decode_window) decode_window;
} lib;
PyObject *s_phase, *s_dim, *s_interleaved, *s_mscale, *s_cuda_stream;  // attribute names

using Shape = std::initializer_list<int64_t>;
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kI32 = at::kInt;

// One call's arguments.  `fine` is false from the first that is not.
struct Args {
  bool fine = true;
  int device = -1;

  // A CUDA tensor on the call's device (that of the first)
  const at::Tensor* tensor(PyObject* o) {
    if (fine && THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.defined() && t.is_cuda() && t.layout() == at::kStrided) {
        if (device < 0) device = t.get_device();
        if (t.get_device() == device) return &t;
      }
    }
    fine = false;
    return nullptr;
  }
  void* any(PyObject* o, at::ScalarType type) {
    const at::Tensor* t = tensor(o);
    if (t && t->scalar_type() == type && t->is_contiguous()) return t->data_ptr();
    fine = false;
    return nullptr;
  }
  void* ptr(PyObject* o, at::ScalarType type, Shape shape) {
    void* p = any(o, type);
    if (fine && THPVariable_Unpack(o).sizes() == at::IntArrayRef(shape)) return p;
    fine = false;
    return nullptr;
  }
  void* optional(PyObject* o, at::ScalarType type, Shape shape) { return o == Py_None ? nullptr : ptr(o, type, shape); }
  template <typename T>
  T* ints(PyObject* o, Shape shape) {
    return static_cast<T*>(ptr(o, sizeof(T) == 8 ? at::kLong : kI32, shape));
  }
  int32_t* optional_ints(PyObject* o, Shape shape) { return o == Py_None ? nullptr : ints<int32_t>(o, shape); }

  int integer(PyObject* o) {
    const long v = fine ? PyLong_AsLong(o) : 0;
    if (fine && ((v == -1 && PyErr_Occurred()) || v < INT32_MIN || v > INT32_MAX)) refuse();
    return (int)v;
  }
  // (sizes that an int cannot hold are refused by the Python path)
  int size(int64_t v) {
    if (v > INT32_MAX) fine = false;
    return (int)v;
  }
  float number(PyObject* o) {
    const double v = fine ? PyFloat_AsDouble(o) : 0;
    if (fine && v == -1 && PyErr_Occurred()) refuse();
    return (float)v;
  }
  PyObject* attribute(PyObject* o, PyObject* name) {  // a new reference
    PyObject* v = fine ? PyObject_GetAttr(o, name) : nullptr;
    if (!v) refuse();
    return v;
  }
  void* stream(PyObject* o) {
    if (!fine) return nullptr;
    if (device != c10::cuda::current_device()) {
      fine = false;
      return nullptr;
    }
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    PyObject* v = attribute(o, s_cuda_stream);
    void* s = v ? PyLong_AsVoidPtr(v) : nullptr;
    if (v && !s && PyErr_Occurred()) refuse();
    Py_XDECREF(v);
    return s;
  }
  void refuse() {
    PyErr_Clear();
    fine = false;
  }
};

// The layout structure of the binding (ctypes), for the length of a call
struct Layout {
  Py_buffer view{};
  const mla_lowbit_layout* l = nullptr;
  Layout(Args& a, PyObject* o) {
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) == 0) {
      if (view.len == (Py_ssize_t)sizeof(mla_lowbit_layout)) l = static_cast<const mla_lowbit_layout*>(view.buf);
    } else {
      view.obj = nullptr;
    }
    if (!l) a.refuse();
  }
  ~Layout() {
    if (view.obj) PyBuffer_Release(&view);
  }
  bool packed() const { return l && l->content_bits != 16; }
};

// A rotation's table and settings; rope None: none
struct Rope {
  const uint64_t* phase = nullptr;
  int dim = 0, interleaved = 0;
  float mscale = 1.f;
  Rope(Args& a, PyObject* o) {
    if (o == Py_None) return;
    PyObject* v = a.attribute(o, s_dim);
    if (v) dim = a.integer(v);
    Py_XDECREF(v);
    v = a.attribute(o, s_interleaved);
    if (v) interleaved = a.integer(v);
    Py_XDECREF(v);
    v = a.attribute(o, s_mscale);
    if (v) mscale = a.number(v);
    Py_XDECREF(v);
    v = a.attribute(o, s_phase);  // (the rope holds it while the call runs)
    if (v) phase = static_cast<const uint64_t*>(a.ptr(v, at::kLong, {dim / 2}));
    Py_XDECREF(v);
  }
};

// A cache's page pool and block table
struct Cache {
  void* pool;
  int64_t pages = 0;
  int32_t* table;
  int seqs = 0, max_pages = 0;
  Cache(Args& a, const Layout& lay, PyObject* page_pool, PyObject* block_table) {
    pool = a.any(page_pool, at::kByte);
    table = static_cast<int32_t*>(a.any(block_table, kI32));
    if (!a.fine) return;
    const at::Tensor &p = THPVariable_Unpack(page_pool), &t = THPVariable_Unpack(block_table);
    if (p.dim() != 2 || t.dim() != 2 || p.size(1) != (int64_t)lib.page_bytes(lay.l)) {
      a.fine = false;
      return;
    }
    pages = p.size(0);
    seqs = a.size(t.size(0));
    max_pages = a.size(t.size(1));
  }
};
struct Buffers {
  void *sink = nullptr, *recent = nullptr;
  Buffers(Args& a, bool used, int seqs, PyObject* sink_buf, PyObject* recent_buf) {
    if (!used) return;
    sink = a.ptr(sink_buf, kBf16, {seqs, 4, 576});
    recent = a.ptr(recent_buf, kBf16, {seqs, 128, 576});
  }
};

int value_type(Args& a, PyObject* out) {  // of an output that may be bf16 or float32
  const at::Tensor* t = a.tensor(out);
  if (t && t->scalar_type() == kBf16) return MLA_LOWBIT_BF16;
  if (t && t->scalar_type() == at::kFloat) return MLA_LOWBIT_FP32;
  a.fine = false;
  return 0;
}
at::ScalarType scalar(int value_type) { return value_type == MLA_LOWBIT_BF16 ? kBf16 : at::kFloat; }

// The call without the interpreter's lock (it may wait for room in a queue)
template <typename F>
PyObject* launched(F call) {  // call must not throw
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// new_lens, seq_lens, block_table, free_pages, free_count, seq_idx, pos, err_word,
// slots, token_start, release, seq_lens_after, free_count_after, stream
PyObject* assign(PyObject* const* v) {
  Args a;
  int32_t* table = static_cast<int32_t*>(a.any(v[2], kI32));
  int32_t* stack = static_cast<int32_t*>(a.any(v[3], kI32));
  int32_t* idx = static_cast<int32_t*>(a.any(v[5], kI32));
  if (!a.fine || THPVariable_Unpack(v[2]).dim() != 2) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(v[2]);
  const int64_t S = t.size(0), n = THPVariable_Unpack(v[5]).numel();
  const int seqs = a.size(S), max_pages = a.size(t.size(1)), pages = a.size(THPVariable_Unpack(v[3]).numel()),
            slots_n = a.size(n);
  const int32_t *new_lens = a.ints<int32_t>(v[0], {S}), *lens = a.ints<int32_t>(v[1], {S}),
                *count = a.ints<int32_t>(v[4], {1}), *release = a.optional_ints(v[10], {S});
  idx = a.ints<int32_t>(v[5], {n});
  int32_t *pos = a.ints<int32_t>(v[6], {n}), *err = a.ints<int32_t>(v[7], {1}), *start = a.optional_ints(v[9], {S + 1}),
          *lens_after = a.ints<int32_t>(v[11] == Py_None ? v[1] : v[11], {S}),
          *count_after = a.ints<int32_t>(v[12] == Py_None ? v[4] : v[12], {1});
  int64_t* slots = static_cast<int64_t*>(a.optional(v[8], at::kLong, {n}));
  void* stream = a.stream(v[13]);
  if (!a.fine) return nullptr;
  return launched([&] {
    return lib.assign(seqs, max_pages, pages, slots_n, new_lens, release, lens, count, table, stack, lens_after, count_after,
                      start, idx, pos, slots, err, stream);
  });
}

// x, pos, rope, offset, norm, weight, eps, out, stream
PyObject* norm_rope(PyObject* const* v) {
  Args a;
  const at::Tensor *x = a.tensor(v[0]), *y = a.tensor(v[7]);
  if (!a.fine) return nullptr;
  const at::ScalarType type = x->scalar_type();
  const int code = type == kBf16 ? MLA_LOWBIT_BF16 : type == at::kHalf ? MLA_LOWBIT_FP16 : MLA_LOWBIT_FP32;
  if ((code == MLA_LOWBIT_FP32 && type != at::kFloat) || x->dim() != 3 || y->scalar_type() != type ||
      y->sizes() != x->sizes() || (x->size(2) > 1 && (x->stride(2) != 1 || y->stride(2) != 1)))
    return nullptr;
  const int n = a.size(x->size(0)), heads = a.size(x->size(1)), dim = a.size(x->size(2));
  const Rope rope(a, v[2]);
  const int32_t* pos = v[2] == Py_None ? nullptr : a.ints<int32_t>(v[1], {n});
  const void* w = a.optional(v[5], type, {dim});
  const int offset = a.integer(v[3]), norm = a.integer(v[4]);
  const float eps = a.number(v[6]);
  void* stream = a.stream(v[8]);
  if (!a.fine) return nullptr;
  const void* xp = x->data_ptr();
  void* yp = y->data_ptr();
  const int64_t xt = x->stride(0), xh = x->stride(1), yt = y->stride(0), yh = y->stride(1);
  return launched([&] {
    return lib.norm_rope(code, n, heads, dim, xp, xt, xh, yp, yt, yh, norm, w, eps, rope.dim, offset, rope.interleaved,
                         rope.phase, rope.mscale, pos, stream);
  });
}

// layout, kv, weight, rope, pos, block_table, page_pool, sink_buf, recent_buf, err_word, eps, seq_idx,
// seq_lens_after, ckv_out, krope_out, stream
PyObject* norm_rope_write(PyObject* const* v) {
  Args a;
  const Layout lay(a, v[0]);
  const Cache c(a, lay, v[6], v[5]);
  const at::Tensor* kv = a.tensor(v[1]);
  if (!a.fine || v[3] == Py_None || kv->scalar_type() != kBf16 || kv->dim() != 2 || kv->size(1) != 576 ||
      kv->stride(1) != 1)
    return nullptr;
  const int n = a.size(kv->size(0));
  const Rope rope(a, v[3]);
  if (rope.dim != 64) return nullptr;
  const void* w = a.optional(v[2], kBf16, {512});
  const int32_t *pos = a.ints<int32_t>(v[4], {n}), *idx = a.optional_ints(v[11], {n}),
                *lens = a.optional_ints(v[12], {c.seqs});
  const Buffers buf(a, lay.packed(), c.seqs, v[7], v[8]);
  void *ckv = a.optional(v[13], kBf16, {n, 512}), *krope = a.optional(v[14], kBf16, {n, 64});
  int32_t* err = a.ints<int32_t>(v[9], {1});
  const float eps = a.number(v[10]);
  void* stream = a.stream(v[15]);
  if (!a.fine) return nullptr;
  const void* rows = kv->data_ptr();
  const int64_t stride = n > 1 ? kv->stride(0) : 576;
  return launched([&] {
    return lib.norm_rope_write(lay.l, n, rows, stride, w, eps, rope.interleaved, rope.phase, rope.mscale, idx, pos, lens,
                               c.seqs, c.table, c.max_pages, c.pool, c.pages, buf.sink, buf.recent, ckv, krope, err,
                               stream);
  });
}

// layout, seq_idx, pos, block_table, page_pool, sink_buf, recent_buf, out, err_word, seq_lens, clear_skipped, stream
PyObject* read(PyObject* const* v) {
  Args a;
  const Layout lay(a, v[0]);
  const Cache c(a, lay, v[4], v[3]);
  const at::Tensor* p = a.tensor(v[2]);
  if (!a.fine) return nullptr;
  const int n = a.size(p->numel());
  const int code = value_type(a, v[7]);
  const int32_t *idx = a.ints<int32_t>(v[1], {n}), *pos = a.ints<int32_t>(v[2], {n}),
                *lens = a.optional_ints(v[9], {c.seqs});
  const Buffers buf(a, lens && lay.packed(), c.seqs, v[5], v[6]);
  void* out = a.ptr(v[7], scalar(code), {n, 576});
  int32_t* err = a.ints<int32_t>(v[8], {1});
  const int clear = a.integer(v[10]) ? MLA_LOWBIT_CLEAR_SKIPPED : 0;
  void* stream = a.stream(v[11]);
  if (!a.fine) return nullptr;
  return launched([&] {
    return lib.read(lay.l, n, idx, pos, c.seqs, lens, c.table, c.max_pages, c.pool, c.pages, buf.sink, buf.recent,
                    code | clear, out, err, stream);
  });
}

// layout, q, page_pool, block_table, seq_lens, sink_buf, recent_buf, out, workspace, err_word, softmax_scale,
// window, sinks, lse, stream
PyObject* decode_window(PyObject* const* v) {
  Args a;
  const Layout lay(a, v[0]);
  const Cache c(a, lay, v[2], v[3]);
  const void* qp = a.any(v[1], kBf16);
  if (!a.fine) return nullptr;
  const at::Tensor& q = THPVariable_Unpack(v[1]);
  if ((q.dim() != 3 && q.dim() != 4) || q.size(-1) != 576 || q.size(0) != c.seqs) return nullptr;
  const bool four = q.dim() == 4;
  const int64_t B = q.size(0), n = four ? q.size(1) : 1, H = q.size(-2);
  const int queries = a.size(n), heads = a.size(H), code = value_type(a, v[7]);
  const int32_t* lens = a.ints<int32_t>(v[4], {B});
  const Buffers buf(a, lay.packed(), c.seqs, v[5], v[6]);
  void* out = four ? a.ptr(v[7], scalar(code), {B, n, H, 512}) : a.ptr(v[7], scalar(code), {B, H, 512});
  float* lse = static_cast<float*>(four ? a.optional(v[13], at::kFloat, {B, n, H}) : a.optional(v[13], at::kFloat, {B, H}));
  void* ws = a.any(v[8], at::kByte);
  int32_t* err = a.ints<int32_t>(v[9], {1});
  const float scale = a.number(v[10]);
  const int window = a.integer(v[11]), sinks = a.integer(v[12]);
  void* stream = a.stream(v[14]);
  if (!a.fine) return nullptr;
  const size_t ws_bytes = (size_t)THPVariable_Unpack(v[8]).numel();
  return launched([&] {
    return lib.decode_window(lay.l, c.seqs, queries, heads, scale, window, sinks, qp, c.pool, c.pages, c.table, c.max_pages,
                             lens, buf.sink, buf.recent, code, out, lse, ws, ws_bytes, err, stream);
  });
}

// data_ptr() and the like may throw; nothing is to leave this file but Python's errors.
template <PyObject* (*call)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  try {
    if (nargs == kArgs && lib.page_bytes) {
      if (PyObject* st = call(args)) return st;
    }
  } catch (...) {
  }
  if (PyErr_Occurred()) PyErr_Clear();
  Py_RETURN_NONE;
}

// bind(page_bytes, assign, norm_rope, norm_rope_write, read, decode_window): the
// library's functions, as addresses
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  void* f[6];
  if (nargs != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    f[i] = PyLong_AsVoidPtr(args[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind takes six addresses");
      return nullptr;
    }
  }
  lib.page_bytes = reinterpret_cast<decltype(lib.page_bytes)>(f[0]);
  lib.assign = reinterpret_cast<decltype(lib.assign)>(f[1]);
  lib.norm_rope = reinterpret_cast<decltype(lib.norm_rope)>(f[2]);
  lib.norm_rope_write = reinterpret_cast<decltype(lib.norm_rope_write)>(f[3]);
  lib.read = reinterpret_cast<decltype(lib.read)>(f[4]);
  lib.decode_window = reinterpret_cast<decltype(lib.decode_window)>(f[5]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", method(bind), METH_FASTCALL, nullptr},
                         {"assign", method(entry<assign, 14>), METH_FASTCALL, nullptr},
                         {"norm_rope", method(entry<norm_rope, 9>), METH_FASTCALL, nullptr},
                         {"norm_rope_write", method(entry<norm_rope_write, 16>), METH_FASTCALL, nullptr},
                         {"read", method(entry<read, 12>), METH_FASTCALL, nullptr},
                         {"decode_window", method(entry<decode_window, 15>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  s_phase = PyUnicode_InternFromString("phase");
  s_dim = PyUnicode_InternFromString("dim");
  s_interleaved = PyUnicode_InternFromString("interleaved");
  s_mscale = PyUnicode_InternFromString("mscale");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return PyModule_Create(&module);
}
