// Python face of the kv_* calls.  They are made once or more a layer for every decoded token, where ctypes and
// checks in Python cost more than the kernels (20 us a call against 5): here a call's arguments are
// checked and passed on in about a microsecond, and outputs come from the caching allocator directly.
// The functions take their arguments by position (api.py names and documents them); a wrong argument
// raises ValueError, the library's status is returned as a number for api.py to raise.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>
#include <utility>

#include "bre.h"

namespace {

using at::Tensor;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::string said(std::initializer_list<int64_t> shape) {
  std::string s = "[";
  for (int64_t d : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(d);
  return s + "]";
}

// The library counts in 32 bits.
int int32(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is outside 32 bits: " + std::to_string(v));
  return (int)v;
}
int integer(PyObject* o, const char* name) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a whole number");
  }
  if (over) refuse(std::string(name) + " is outside 32 bits");
  return int32(v, name);
}

// An owned reference.
struct Ref {
  PyObject* o;
  explicit Ref(PyObject* p) : o(p) {}
  Ref(Ref&& r) : o(r.o) { r.o = nullptr; }
  ~Ref() { Py_XDECREF(o); }
  void* data() const { return THPVariable_Unpack(o).data_ptr(); }
};

PyObject *name_pages, *name_bounds, *name_bound_exp;   // interned by the module's start

// A KvCache as its fields are at the time of the call: they may have been assigned since it was made (a cache that
// grows), and a copy has tensors of its own.  Nothing of it is kept from one call for the next.
struct Cache {
  Ref pages, bounds, bound_exp;
  int n, heads, dim;

  static Ref field(PyObject* cache, PyObject* name) {
    PyObject* o = PyObject_GetAttr(cache, name);
    if (!o) {
      PyErr_Clear();
      refuse("not a cache");
    }
    return Ref(o);
  }
  explicit Cache(PyObject* cache)
      : pages(field(cache, name_pages)), bounds(field(cache, name_bounds)), bound_exp(field(cache, name_bound_exp)) {
    const Tensor &p = tensor(pages.o, "pages"), &b = tensor(bounds.o, "bounds"), &e = tensor(bound_exp.o, "bound_exp");
    if (b.dim() != 4 || b.size(2) != 2) refuse("bounds must be [n_pages, n_kv_heads, 2, head_dim]");
    n = int32(b.size(0), "n_pages"), heads = int32(b.size(1), "n_kv_heads"), dim = int32(b.size(3), "head_dim");
    if (p.sizes() != at::IntArrayRef({n, heads, 128 * (dim + 1LL)}) || e.sizes() != at::IntArrayRef({n, heads}))
      refuse("pages, bounds and bound_exp do not belong together");
    if (p.scalar_type() != at::kByte || b.scalar_type() != at::kChar || e.scalar_type() != at::kChar)
      refuse("pages must be uint8, bounds and bound_exp int8");
    for (const Tensor* t : {&p, &b, &e})
      if (!t->is_cuda() || !t->is_contiguous()) refuse("pages, bounds and bound_exp must be contiguous CUDA tensors");
    device(nullptr, 0);
  }
  // The cache's device; refuses tensors among a call's other arguments that are not there.
  c10::Device device(PyObject* const* a, Py_ssize_t n) const {
    const c10::Device d = THPVariable_Unpack(pages.o).device();
    auto there = [&](PyObject* o) {
      const c10::Device x = THPVariable_Unpack(o).device();
      if (x != d) refuse("all tensors must be on the CUDA device of the cache's pages, " + d.str() + ": there is one on " + x.str());
    };
    there(bounds.o);
    there(bound_exp.o);
    for (Py_ssize_t i = 0; i < n; ++i)   // (THPVariable_Check takes long over what is no tensor)
      if (a[i] != Py_None && !PyLong_CheckExact(a[i]) && !PyFloat_CheckExact(a[i]) && THPVariable_Check(a[i])) there(a[i]);
    return d;
  }
  bre_kv_cache native() const {
    return {pages.data(), static_cast<int8_t*>(bounds.data()), static_cast<int8_t*>(bound_exp.data()), n, heads, dim};
  }
};

// A contiguous CUDA tensor of this type and shape.
template <typename P = void>
P* like(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_cuda() || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " CUDA tensor " + said(shape));
  return static_cast<P*>(t.data_ptr());
}

// Row stride (elements) of [T, heads, D] BF16 rows (or their 16-bit patterns), which may be a slice of wider
// rows; heads < 0: any number, returned in *n_heads.
const void* rows(PyObject* o, const char* name, int64_t T, int64_t heads, int64_t D, int64_t* stride, int* n_heads = nullptr) {
  const Tensor& t = tensor(o, name);
  if (t.dim() != 3 || t.size(0) != T || t.size(2) != D || (heads >= 0 && t.size(1) != heads))
    refuse(std::string(name) + " must be " + said({T, heads, D}));
  if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != D))
    refuse(std::string(name) + ": a token's heads must follow one another without gaps");
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.element_size() != 2 || t.scalar_type() == at::kHalf) refuse(std::string(name) + " must be bfloat16");
  *stride = T > 1 ? t.stride(0) : (t.size(1) * D + 7) / 8 * 8;
  if (n_heads) *n_heads = int32(t.size(1), "the number of heads");
  return t.data_ptr();
}

// A call's cache, tokens and stream.  The cache's device, which every tensor among the arguments must be on, is the
// current one while the call lasts (streams, attributes and launches go by it).
struct Call {
  Cache cache;
  c10::Device device;
  c10::cuda::OptionalCUDAGuard guard;
  bre_kv_cache c;
  const int32_t *seq, *pos, *table;
  int T, B, N;
  bre_stream_t stream;
  std::optional<c10::cuda::CUDAStream> current;   // where it is not the call's
  int32_t* err;

  // a: the call's n arguments, of which the first is the cache, `tokens` and the two after it seq, pos and table, the
  // last but one dev_err and the last the stream
  Call(PyObject* const* a, Py_ssize_t n, int tokens)
      : cache(a[0]), device(cache.device(a + 1, n - 1)) {
    PyObject *const seq_o = a[tokens], *const pos_o = a[tokens + 1], *const table_o = a[tokens + 2];
    PyObject *const err_o = a[n - 2], *const stream_o = a[n - 1];
    const Tensor& s = tensor(seq_o, "seq");
    const Tensor& t = tensor(table_o, "table");
    if (s.dim() != 1 || t.dim() != 2) refuse("seq must be [T] and table [B, N]");
    T = int32(s.size(0), "T"), B = int32(t.size(0), "B"), N = int32(t.size(1), "N");
    if (c10::cuda::current_device() != device.index()) guard.set_device(device);   // (a guard costs about a microsecond)
    c = cache.native();
    seq = like<int32_t>(seq_o, "seq", at::kInt, {T});
    pos = like<int32_t>(pos_o, "pos", at::kInt, {T});
    table = like<int32_t>(table_o, "table", at::kInt, {B, N});
    err = err_o == Py_None ? nullptr : like<int32_t>(err_o, "dev_err", at::kInt, {1});
    const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(device.index());
    cudaStream_t on = now.stream();
    if (stream_o != Py_None) {
      on = static_cast<cudaStream_t>(PyLong_AsVoidPtr(stream_o));
      if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("not a stream");
      }
      if (on != now.stream()) current = now;
    }
    stream = reinterpret_cast<bre_stream_t>(on);
  }
  // The caller's output, or a new one.  For a call on another stream than the current one it is allocated there:
  // memory of the current stream may be in use by work that the other stream does not wait for.  The
  // caller, who is on the current stream, is a user of it too.
  Ref output(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    if (o == Py_None) {
      if (!current) return Ref(THPVariable_Wrap(at::detail::empty_cuda(at::IntArrayRef(shape), type, device, std::nullopt)));
      const c10::cuda::CUDAStreamGuard there(
          c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream), device.index()));
      const Tensor t = at::detail::empty_cuda(at::IntArrayRef(shape), type, device, std::nullopt);
      t.record_stream(*current);
      return Ref(THPVariable_Wrap(t));
    }
    like(o, name, type, shape);
    Py_INCREF(o);
    return Ref(o);
  }
};

// The caller's workspace (no call needs one).
struct Workspace {
  void* p = nullptr;
  size_t n = 0;
  Workspace(PyObject* o) {
    if (o == Py_None) return;
    const Tensor& t = tensor(o, "ws");
    if (!t.is_cuda() || !t.is_contiguous() || t.scalar_type() != at::kByte) refuse("ws must be a contiguous uint8 CUDA tensor");
    p = t.data_ptr();
    n = (size_t)t.numel();
  }
};

// (status, first output, second output)
PyObject* answer(bre_status st, Ref& a, Ref& b) {
  PyObject* r = PyTuple_New(3);
  if (!r) throw std::bad_alloc();
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(st));
  PyTuple_SET_ITEM(r, 1, std::exchange(a.o, nullptr));
  PyTuple_SET_ITEM(r, 2, std::exchange(b.o, nullptr));
  return r;
}

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  try {
    if (given != wanted) refuse("wrong number of arguments");
    return f();
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {   // cache k v seq pos table dev_err stream
  return guarded(n, 8, [&] {
    const Call call(a, n, 3);
    int64_t ks, vs;
    const void* k = rows(a[1], "k", call.T, call.c.n_kv_heads, call.c.head_dim, &ks);
    const void* v = rows(a[2], "v", call.T, call.c.n_kv_heads, call.c.head_dim, &vs);
    return PyLong_FromLong(kv_append(&call.c, k, v, ks, vs, call.seq, call.pos, call.T, call.table, call.B, call.N, call.err,
                                     call.stream));
  });
}

PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {   // cache seq pos table k_out v_out dev_err stream
  return guarded(n, 8, [&] {
    const Call call(a, n, 1);
    Ref k = call.output(a[4], "k_out", at::kBFloat16, {call.T, call.c.n_kv_heads, call.c.head_dim});
    Ref v = call.output(a[5], "v_out", at::kBFloat16, {call.T, call.c.n_kv_heads, call.c.head_dim});
    const bre_status st =
        kv_read(&call.c, call.seq, call.pos, call.T, call.table, call.B, call.N, k.data(), v.data(), call.err, call.stream);
    return answer(st, k, v);
  });
}

// cache q seq pos table k n_sink n_local ws ids scores dev_err stream
PyObject* py_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const int k = integer(a[5], "k"), sink = integer(a[6], "n_sink"), local = integer(a[7], "n_local");
    const Call call(a, n, 2);
    const int H = call.c.n_kv_heads;
    if (k < 0) refuse("k must not be negative");
    int64_t qs;
    int Hq;
    const void* q = rows(a[1], "q", call.T, -1, call.c.head_dim, &qs, &Hq);
    const Workspace ws(a[8]);
    Ref ids = call.output(a[9], "ids", at::kInt, {call.T, H, k});
    Ref sc = call.output(a[10], "scores", at::kFloat, {call.T, H, k});
    const bre_status st = kv_select(&call.c, q, qs, Hq, call.seq, call.pos, call.T, call.table, call.B, call.N, k, sink, local,
                                    static_cast<int32_t*>(ids.data()), static_cast<float*>(sc.data()), ws.p, ws.n, call.err,
                                    call.stream);
    return answer(st, ids, sc);
  });
}

// cache q seq pos table ids scale ws out lse dev_err stream
PyObject* py_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const Call call(a, n, 2);
    const int H = call.c.n_kv_heads, D = call.c.head_dim;
    int64_t qs;
    int Hq;
    const void* q = rows(a[1], "q", call.T, -1, D, &qs, &Hq);
    const Tensor& id = tensor(a[5], "ids");
    if (id.dim() != 3) refuse("ids must be [T, n_kv_heads, k]");
    const int k = int32(id.size(2), "k");
    const int32_t* ids = like<int32_t>(a[5], "ids", at::kInt, {call.T, H, k});
    const double scale = a[6] == Py_None ? std::pow((double)D, -0.5) : PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("scale must be a number");
    }
    const Workspace ws(a[7]);
    Ref out = call.output(a[8], "out", at::kBFloat16, {call.T, Hq, D});
    Ref lse = call.output(a[9], "lse", at::kFloat, {call.T, Hq});
    const bre_status st = kv_attend(&call.c, q, qs, Hq, call.seq, call.pos, call.T, call.table, call.B, call.N, ids, k,
                                    (float)scale, out.data(), static_cast<float*>(lse.data()), ws.p, ws.n, call.err, call.stream);
    return answer(st, out, lse);
  });
}

// cache -> None: refuses what is no cache
PyObject* py_check(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject* {
    const Cache c(a[0]);
    Py_RETURN_NONE;
  });
}

PyMethodDef methods[] = {
    {"check", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_check)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_append)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_read)), METH_FASTCALL, nullptr},
    {"select", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_select)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_attend)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv() {
  name_pages = PyUnicode_InternFromString("pages");
  name_bounds = PyUnicode_InternFromString("bounds");
  name_bound_exp = PyUnicode_InternFromString("bound_exp");
  return name_pages && name_bounds && name_bound_exp ? PyModule_Create(&module) : nullptr;
}
