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

double number(PyObject* o, const char* name, double unless) {
  const double v = o == Py_None ? unless : PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return v;
}

// An owned reference.
struct Ref {
  PyObject* o;
  explicit Ref(PyObject* p) : o(p) {}
  Ref(Ref&& r) : o(r.o) { r.o = nullptr; }
  Ref& operator=(Ref&& r) {
    std::swap(o, r.o);
    return *this;
  }
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

// Where a call runs: its device, which is the current one while the call lasts (streams, attributes and launches go by
// it), and its stream.
struct Where {
  c10::Device device{c10::kCUDA};
  c10::cuda::OptionalCUDAGuard guard;
  bre_stream_t stream = nullptr;
  std::optional<c10::cuda::CUDAStream> current;   // where it is not the call's

  void enter(c10::Device d, PyObject* stream_o) {
    device = d;
    if (c10::cuda::current_device() != device.index()) guard.set_device(device);   // (a guard costs about a microsecond)
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
  // A new tensor.  For a call on another stream than the current one it is allocated there: memory of the current
  // stream may be in use by work that the other stream does not wait for.  The caller, who is on the current stream, is a
  // user of it too.
  Ref fresh(at::ScalarType type, at::IntArrayRef shape) const {
    if (!current) return Ref(THPVariable_Wrap(at::detail::empty_cuda(shape, type, device, std::nullopt)));
    const c10::cuda::CUDAStreamGuard there(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream), device.index()));
    const Tensor t = at::detail::empty_cuda(shape, type, device, std::nullopt);
    t.record_stream(*current);
    return Ref(THPVariable_Wrap(t));
  }
  // The caller's output, or a new one.
  Ref output(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    if (o == Py_None) return fresh(type, shape);
    like(o, name, type, shape);
    Py_INCREF(o);
    return Ref(o);
  }
};

// A call on a cache's pages: the cache, the page table and, where it is for tokens, these.  Every tensor among the arguments
// must be on the cache's device.  Sizes are looked at before the device is.
struct Call : Where {
  Cache cache;
  bre_kv_cache c;
  const int32_t *seq = nullptr, *pos = nullptr, *table;
  int T = 0, B, N;
  int32_t* err;

  // a: the call's n arguments, of which the first is the cache, the last but one dev_err and the last the stream;
  // tokens >= 0: where seq and pos are
  Call(PyObject* const* a, Py_ssize_t n, int table_at, int tokens) : cache(a[0]) {
    const c10::Device on = cache.device(a + 1, n - 1);
    const Tensor& t = tensor(a[table_at], "table");
    if ((tokens >= 0 && tensor(a[tokens], "seq").dim() != 1) || t.dim() != 2) refuse("seq must be [T] and table [B, N]");
    if (tokens >= 0) T = int32(tensor(a[tokens], "seq").size(0), "T");
    B = int32(t.size(0), "B"), N = int32(t.size(1), "N");
    enter(on, a[n - 1]);
    c = cache.native();
    if (tokens >= 0) {
      seq = like<int32_t>(a[tokens], "seq", at::kInt, {T});
      pos = like<int32_t>(a[tokens + 1], "pos", at::kInt, {T});
    }
    table = like<int32_t>(a[table_at], "table", at::kInt, {B, N});
    err = a[n - 2] == Py_None ? nullptr : like<int32_t>(a[n - 2], "dev_err", at::kInt, {1});
  }
};

// The caller's workspace.
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
  // One of `need` bytes where the caller gave none: it lives as long as the call, and its memory is used again only by
  // work that is ordered after the call's.
  Workspace(PyObject* o, const Where& at, size_t need) : Workspace(o) {
    if (o != Py_None || need == 0) return;
    own.emplace(at.fresh(at::kByte, {(int64_t)need}));
    p = own->data();
    n = need;
  }

 private:
  std::optional<Ref> own;
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
    const Call call(a, n, 5, 3);
    int64_t ks, vs;
    const void* k = rows(a[1], "k", call.T, call.c.n_kv_heads, call.c.head_dim, &ks);
    const void* v = rows(a[2], "v", call.T, call.c.n_kv_heads, call.c.head_dim, &vs);
    return PyLong_FromLong(kv_append(&call.c, k, v, ks, vs, call.seq, call.pos, call.T, call.table, call.B, call.N, call.err,
                                     call.stream));
  });
}

PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {   // cache seq pos table k_out v_out dev_err stream
  return guarded(n, 8, [&] {
    const Call call(a, n, 3, 1);
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
    const Call call(a, n, 4, 2);
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
    const Call call(a, n, 4, 2);
    const int H = call.c.n_kv_heads, D = call.c.head_dim;
    int64_t qs;
    int Hq;
    const void* q = rows(a[1], "q", call.T, -1, D, &qs, &Hq);
    const Tensor& id = tensor(a[5], "ids");
    if (id.dim() != 3) refuse("ids must be [T, n_kv_heads, k]");
    const int k = int32(id.size(2), "k");
    const int32_t* ids = like<int32_t>(a[5], "ids", at::kInt, {call.T, H, k});
    const double scale = number(a[6], "scale", std::pow((double)D, -0.5));
    const Workspace ws(a[7]);
    Ref out = call.output(a[8], "out", at::kBFloat16, {call.T, Hq, D});
    Ref lse = call.output(a[9], "lse", at::kFloat, {call.T, Hq});
    const bre_status st = kv_attend(&call.c, q, qs, Hq, call.seq, call.pos, call.T, call.table, call.B, call.N, ids, k,
                                    (float)scale, out.data(), static_cast<float*>(lse.data()), ws.p, ws.n, call.err, call.stream);
    return answer(st, out, lse);
  });
}

// cache q seq pos table start mask scale ws out lse dev_err stream
PyObject* py_attend_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Call call(a, n, 4, 2);
    const int H = call.c.n_kv_heads, D = call.c.head_dim;
    int64_t qs;
    int Hq;
    const void* q = rows(a[1], "q", call.T, -1, D, &qs, &Hq);
    const int32_t* start = nullptr;
    const uint64_t* mask = nullptr;
    int words = 0;
    if (a[6] != Py_None) {
      if (a[5] == Py_None) refuse("mask needs start");
      const Tensor& m = tensor(a[6], "mask");
      if (m.dim() != 2) refuse("mask must be [T, words]");
      words = int32(m.size(1), "words");
      mask = reinterpret_cast<const uint64_t*>(like<int64_t>(a[6], "mask", at::kLong, {call.T, words}));
    }
    if (a[5] != Py_None) start = like<int32_t>(a[5], "start", at::kInt, {call.B});
    const double scale = number(a[7], "scale", std::pow((double)D, -0.5));
    const Workspace ws(a[8], call, kv_attend_tree_workspace(call.T, Hq, H, D));
    Ref out = call.output(a[9], "out", at::kBFloat16, {call.T, Hq, D});
    Ref lse = call.output(a[10], "lse", at::kFloat, {call.T, Hq});
    const bre_status st = kv_attend_tree(&call.c, q, qs, Hq, call.seq, call.pos, call.T, call.table, call.B, call.N, start, mask,
                                         words, (float)scale, out.data(), static_cast<float*>(lse.data()), ws.p, ws.n, call.err,
                                         call.stream);
    return answer(st, out, lse);
  });
}

// q k pos turns gain offset interleaved backward q_out k_out stream
PyObject* py_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const Tensor &q = tensor(a[0], "q"), &p = tensor(a[2], "pos"), &w = tensor(a[3], "turns");
    if (q.dim() != 3 || p.dim() != 1 || w.dim() != 1) refuse("q must be [T, n_heads, D], pos [T] and turns [n_pairs]");
    if (!q.is_cuda()) refuse("q must be a CUDA tensor");
    for (int i : {1, 2, 3, 8, 9})
      if (a[i] != Py_None && tensor(a[i], "k, pos, turns, q_out and k_out").device() != q.device())
        refuse("all tensors must be on q's device, " + q.device().str());
    const int T = int32(q.size(0), "T"), pairs = int32(w.size(0), "n_pairs"), offset = integer(a[5], "offset");
    Where at;
    at.enter(q.device(), a[10]);
    const int64_t D = q.size(2);
    const int32_t* pos = like<int32_t>(a[2], "pos", at::kInt, {T});
    const uint64_t* turns = reinterpret_cast<const uint64_t*>(like<int64_t>(a[3], "turns", at::kLong, {pairs}));
    const double gain = number(a[4], "gain", 1.0);
    int64_t qs, ks = 0, qos, kos = 0;
    int Hq, Hk = 0;
    const void *qp = rows(a[0], "q", T, -1, D, &qs, &Hq), *kp = nullptr;
    auto out = [&](PyObject* o, const char* name, int heads, int64_t* stride) {
      Ref r = o == Py_None ? at.fresh(at::kBFloat16, {T, heads, D}) : (Py_INCREF(o), Ref(o));
      rows(r.o, name, T, heads, D, stride);
      return r;
    };
    Ref qo = out(a[8], "q_out", Hq, &qos), ko(nullptr);
    if (a[1] != Py_None) {
      kp = rows(a[1], "k", T, -1, D, &ks, &Hk);
      ko = out(a[9], "k_out", Hk, &kos);
    } else {
      if (a[9] != Py_None) refuse("k_out without k");
      Py_INCREF(Py_None);
      ko = Ref(Py_None);
    }
    const int turned = PyObject_IsTrue(a[6]), back = PyObject_IsTrue(a[7]);
    if (turned < 0 || back < 0) {
      PyErr_Clear();
      refuse("interleaved and backward must be truth values");
    }
    const bre_status st = kv_rotate(qp, qs, Hq, kp, ks, Hk, int32(D, "D"), pos, T, turns, pairs, (float)gain, offset, turned, back,
                                    qo.data(), qos, kp ? ko.data() : nullptr, kos, at.stream);
    return answer(st, qo, ko);
  });
}

// cache table start nodes count length dev_err stream
PyObject* py_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Call call(a, n, 1, -1);
    const Tensor& nd = tensor(a[3], "nodes");
    if (nd.dim() != 2) refuse("nodes must be [B, A]");
    const int A = int32(nd.size(1), "A");
    const int32_t* start = like<int32_t>(a[2], "start", at::kInt, {call.B});
    const int32_t* nodes = like<int32_t>(a[3], "nodes", at::kInt, {call.B, A});
    const int32_t* count = like<int32_t>(a[4], "count", at::kInt, {call.B});
    Ref length = call.output(a[5], "length", at::kInt, {call.B}), none(nullptr);
    Py_INCREF(Py_None);
    none = Ref(Py_None);
    const bre_status st = kv_compact(&call.c, call.table, call.B, call.N, start, nodes, A, count,
                                     static_cast<int32_t*>(length.data()), call.err, call.stream);
    return answer(st, length, none);
  });
}

// cache refs table parent length dev_err stream
PyObject* py_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Call call(a, n, 2, -1);
    int32_t* refs = like<int32_t>(a[1], "refs", at::kInt, {call.c.n_pages});
    const int32_t* parent = like<int32_t>(a[3], "parent", at::kInt, {call.B});
    const int32_t* length = like<int32_t>(a[4], "length", at::kInt, {call.B});
    return PyLong_FromLong(kv_fork(&call.c, refs, const_cast<int32_t*>(call.table), call.B, call.N, parent, length, call.err,
                                   call.stream));
  });
}

// cache refs table start end ws dev_err stream
PyObject* py_resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Call call(a, n, 2, -1);
    int32_t* refs = like<int32_t>(a[1], "refs", at::kInt, {call.c.n_pages});
    const int32_t* start = like<int32_t>(a[3], "start", at::kInt, {call.B});
    const int32_t* end = like<int32_t>(a[4], "end", at::kInt, {call.B});
    const Workspace ws(a[5], call, kv_resize_workspace(call.c.n_pages, call.B, call.N));
    return PyLong_FromLong(kv_resize(&call.c, refs, const_cast<int32_t*>(call.table), call.B, call.N, start, end, ws.p, ws.n,
                                     call.err, call.stream));
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
    {"attend_tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_attend_tree)), METH_FASTCALL, nullptr},
    {"rotate", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_rotate)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_compact)), METH_FASTCALL, nullptr},
    {"fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_fork)), METH_FASTCALL, nullptr},
    {"resize", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_resize)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv() {
  name_pages = PyUnicode_InternFromString("pages");
  name_bounds = PyUnicode_InternFromString("bounds");
  name_bound_exp = PyUnicode_InternFromString("bound_exp");
  return name_pages && name_bounds && name_bound_exp ? PyModule_Create(&module) : nullptr;
}
