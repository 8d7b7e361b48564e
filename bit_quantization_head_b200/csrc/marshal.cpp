// The binding's side of the calls around the cache (module _marshal): checks torch tensors,
// takes their pointers and the current stream, calls the library and returns its status.
// Argument marshalling only; kvtc.py turns a status into an exception.  Compiled because the
// smallest calls are bound by the host: the same checks in Python took 5 to 7 us of a call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstring>
#include <exception>
#include <string>

#include "kvtc.h"

namespace {

struct {
  decltype(&kvtc_step_tables) step_tables;
  decltype(&kvtc_rope) rope;
  decltype(&kvtc_raw_append) raw_append;
  decltype(&kvtc_raw_decode_attention) raw_decode;
  decltype(&kvtc_raw_cross_attention) raw_cross;
} fns;

// A refused argument: the Python exception and its message.
struct Refused : std::exception {
  PyObject* type;
  std::string text;
  Refused(PyObject* t, std::string s) : type(t), text(std::move(s)) {}
};
// A Python exception that is set already.
struct Raised : std::exception {};

[[noreturn]] void value_error(std::string text) { throw Refused(PyExc_ValueError, std::move(text)); }
[[noreturn]] void type_error(std::string text) { throw Refused(PyExc_TypeError, std::move(text)); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
int small_integer(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " out of range");
  return static_cast<int>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised();
  return p;
}
// Sizes that the library takes as int.
int count(int64_t n, const char* name) {
  if (n > INT32_MAX) value_error(std::string(name) + " has too many elements");
  return static_cast<int>(n);
}

std::string shape_text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

void on_device(const at::Tensor& t, int dev, const char* name) {
  if (!t.is_cuda() || t.get_device() != dev) value_error(std::string(name) + " must be on the current CUDA device");
}
// Index of the device of a tensor, which must be the current one.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
    value_error(std::string(name) + " must be on the current CUDA device");
  return static_cast<int>(t.get_device());
}

void of_type(const at::Tensor& t, at::ScalarType dtype, const char* name) {
  if (t.scalar_type() != dtype)
    type_error(std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
}
// Pointer of a contiguous tensor of n elements (n < 0: any number).
void* buffer(PyObject* o, at::ScalarType dtype, const char* name, int dev, int64_t n) {
  const at::Tensor& t = tensor(o, name);
  on_device(t, dev, name);
  of_type(t, dtype, name);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  if (n >= 0 && t.numel() != n)
    value_error(std::string(name) + " must have " + std::to_string(n) + " elements, got " + std::to_string(t.numel()));
  return t.data_ptr();
}
void* buffer_like(PyObject* o, const at::Tensor& like, const char* name, int dev) {
  const at::Tensor& t = tensor(o, name);
  on_device(t, dev, name);
  of_type(t, like.scalar_type(), name);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  if (t.sizes() != like.sizes())
    value_error(std::string(name) + " must have shape " + shape_text(like.sizes()) + ", got " + shape_text(t.sizes()));
  return t.data_ptr();
}
// A workspace of any type: its pointer and bytes.
void* workspace(PyObject* o, int dev, uint64_t& bytes) {
  const at::Tensor& t = tensor(o, "workspace");
  on_device(t, dev, "workspace");
  if (!t.is_contiguous()) value_error("workspace must be contiguous");
  bytes = t.nbytes();
  return t.data_ptr();
}

// Rows [n_tok][heads][128] whose heads and elements are dense (a slice of a fused projection
// passes as it is).
struct Rows {
  const void* p = nullptr;
  int64_t stride = 0;
  int heads = 0;
};
Rows rows(const at::Tensor& t, at::ScalarType dtype, const char* name, int dev, int64_t n_tok) {
  on_device(t, dev, name);
  of_type(t, dtype, name);
  if (t.dim() != 3 || t.size(2) != 128 || t.size(0) != n_tok)
    value_error(std::string(name) + " must have shape [n_tok][heads][128], got " + shape_text(t.sizes()));
  if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != 128))
    value_error(std::string(name) + ": heads and elements must be dense");
  Rows r;
  r.p = t.data_ptr();
  r.heads = count(t.size(1), name);
  r.stride = n_tok > 1 ? t.stride(0) : std::max<int64_t>(1, t.size(1) * 128);
  return r;
}
kvtc_dtype code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return KVTC_F32;
    case at::kBFloat16: return KVTC_BF16;
    case at::kHalf: return KVTC_F16;
    default: type_error(std::string("unsupported dtype ") + c10::toString(t));
  }
}
const int32_t* positions(const kvtc_rope_desc* d, PyObject* o, int64_t n_tok, int dev) {
  const at::Tensor& t = tensor(o, "positions");
  if (t.dim() < 1 || t.numel() != d->n_axes * n_tok || t.size(-1) != n_tok)
    value_error("positions must have shape [" + std::to_string(d->n_axes) + "][" + std::to_string(n_tok) + "]");
  return static_cast<const int32_t*>(buffer(o, at::kInt, "positions", dev, -1));
}

void* stream_of(PyObject* o, int dev) {
  return o == Py_None ? c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream() : address(o);
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(static_cast<long>(f()));
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
template <typename F>
kvtc_status without_gil(F f) {
  kvtc_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  return st;
}

// (cached_lens, new_lens, page_ring, ring_state, block_table, seq_lens, cu_seqlens, slot_map,
//  positions, ring_state_out, workspace, status or None, stream or None)
PyObject* step_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const at::Tensor& cached = tensor(a[0], "cached_lens");
    const int dev = device_of(cached, "cached_lens");
    const int64_t seqs = cached.numel(), rows = tensor(a[7], "slot_map").numel();
    const at::Tensor& table = tensor(a[4], "block_table");
    if (table.dim() != 2) value_error("block_table must have shape [n_seq][max_pages]");
    const int64_t max_pages = table.size(1);
    uint64_t ws_bytes = 0;
    auto i32 = [&](int i, const char* name, int64_t count) {
      return static_cast<int32_t*>(buffer(a[i], at::kInt, name, dev, count));
    };
    const int32_t *c = i32(0, "cached_lens", seqs), *f = i32(1, "new_lens", seqs);
    int32_t* ring = i32(2, "page_ring", -1);
    const int32_t* state = i32(3, "ring_state", 2);
    int32_t *tab = i32(4, "block_table", seqs * max_pages), *seq = i32(5, "seq_lens", seqs);
    int32_t* cu = i32(6, "cu_seqlens", seqs + 1);
    int64_t* slots = static_cast<int64_t*>(buffer(a[7], at::kLong, "slot_map", dev, -1));
    int32_t *pos = i32(8, "positions", rows), *out = i32(9, "ring_state_out", 2);
    void* ws = workspace(a[10], dev, ws_bytes);
    if (ws_bytes < 16) value_error("workspace must hold 16 bytes");
    int32_t* status = a[11] == Py_None ? nullptr : i32(11, "status", -1);
    void* stream = stream_of(a[12], dev);
    const int n_seq = count(seqs, "cached_lens"), capacity = count(tensor(a[2], "page_ring").numel(), "page_ring");
    const int pages = count(max_pages, "block_table"), n_rows = count(rows, "slot_map");
    return without_gil([&] {
      return fns.step_tables(c, f, n_seq, ring, capacity, state, tab, pages, seq, cu, slots, pos, n_rows, out, ws, status,
                             stream);
    });
  });
}

// (address of the description, q or None, k or None, positions, q_out, k_out, inverse, stream
//  or None)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const auto* d = static_cast<const kvtc_rope_desc*>(address(a[0]));
    const bool has_q = a[1] != Py_None, has_k = a[2] != Py_None;
    if (!has_q && !has_k) value_error("q or k must be given");
    const at::Tensor& ref = tensor(a[has_q ? 1 : 2], has_q ? "q" : "k");
    const at::ScalarType dtype = ref.scalar_type();
    const kvtc_dtype type = code(dtype);
    const int dev = device_of(ref, has_q ? "q" : "k");
    if (ref.dim() < 1) value_error("q and k must have shape [n_tok][heads][128]");
    const int64_t n_tok = ref.size(0);
    Rows q, k;
    void *qo = nullptr, *ko = nullptr;
    if (has_q) {
      q = rows(ref, dtype, "q", dev, n_tok);
      qo = buffer_like(a[4], ref, "q_out", dev);
    }
    if (has_k) {
      const at::Tensor& kt = tensor(a[2], "k");
      k = rows(kt, dtype, "k", dev, n_tok);
      ko = buffer_like(a[5], kt, "k_out", dev);
    }
    const int32_t* pos = positions(d, a[3], n_tok, dev);
    const int inverse = PyObject_IsTrue(a[6]);
    if (inverse < 0) throw Raised();
    void* stream = stream_of(a[7], dev);
    const int tokens = count(n_tok, "q");
    return without_gil([&] {
      return fns.rope(d, q.p, q.stride, q.heads, k.p, k.stride, k.heads, type, pos, tokens, inverse, qo, ko, stream);
    });
  });
}

// (address of the cache, its pool, layer, k, v, slot_map, address of the description or None,
//  positions, q or None, q_out, stream or None)
PyObject* raw_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const auto* cache = static_cast<const kvtc_raw_cache*>(address(a[0]));
    const at::Tensor& pool = tensor(a[1], "the cache");
    const at::ScalarType dtype = pool.scalar_type();
    const int dev = device_of(pool, "the cache"), layer = small_integer(a[2], "layer");
    const at::Tensor& kt = tensor(a[3], "k");
    if (kt.dim() < 1) value_error("k must have shape [n_tok][heads][128]");
    const int64_t n_tok = kt.size(0);
    const Rows k = rows(kt, dtype, "k", dev, n_tok), v = rows(tensor(a[4], "v"), dtype, "v", dev, n_tok);
    if (k.heads != cache->n_kv_heads || v.heads != cache->n_kv_heads)
      value_error("k and v must have " + std::to_string(cache->n_kv_heads) + " heads");
    const auto* slots = static_cast<const int64_t*>(buffer(a[5], at::kLong, "slot_map", dev, n_tok));
    const kvtc_rope_desc* d = a[6] == Py_None ? nullptr : static_cast<const kvtc_rope_desc*>(address(a[6]));
    if (d && a[7] == Py_None) value_error("rope needs positions");
    const int32_t* pos = d ? positions(d, a[7], n_tok, dev) : nullptr;
    Rows q;
    void* qo = nullptr;
    if (a[8] != Py_None) {
      const at::Tensor& qt = tensor(a[8], "q");
      q = rows(qt, dtype, "q", dev, n_tok);
      qo = buffer_like(a[9], qt, "q_out", dev);
    }
    void* stream = stream_of(a[10], dev);
    const int tokens = count(n_tok, "k");
    return without_gil([&] {
      return fns.raw_append(cache, layer, k.p, k.stride, v.p, v.stride, slots, tokens, d, pos, q.p, q.stride, q.heads, qo,
                            stream);
    });
  });
}

// Query rows [rows][n_q_heads][128] of the cache's type.
const at::Tensor& queries(PyObject* o, const at::Tensor& pool, int dev, int64_t n_rows) {
  const at::Tensor& q = tensor(o, "q");
  if (q.dim() != 3 || (n_rows >= 0 && q.size(0) != n_rows) || q.size(2) != 128)
    value_error("q must have shape [rows][n_q_heads][128], got " + shape_text(q.sizes()));
  (void)buffer(o, pool.scalar_type(), "q", dev, -1);
  return q;
}

// (address of the cache, its pool, layer, q, seq_lens, max_seq_len, out, workspace, scale,
//  stream or None)
PyObject* raw_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const auto* cache = static_cast<const kvtc_raw_cache*>(address(a[0]));
    const at::Tensor& pool = tensor(a[1], "the cache");
    const int dev = device_of(pool, "the cache"), layer = small_integer(a[2], "layer");
    const at::Tensor& q = queries(a[3], pool, dev, cache->n_seq);
    const auto* lens = static_cast<const int32_t*>(buffer(a[4], at::kInt, "seq_lens", dev, cache->n_seq));
    const int max_len = small_integer(a[5], "max_seq_len");
    void* out = buffer_like(a[6], q, "out", dev);
    uint64_t bytes = 0;
    void* ws = workspace(a[7], dev, bytes);
    const float scale = static_cast<float>(number(a[8]));
    void* stream = stream_of(a[9], dev);
    const int heads = count(q.size(1), "q");
    const void* qp = q.data_ptr();
    return without_gil([&] {
      return fns.raw_decode(cache, layer, qp, heads, lens, max_len, scale, out, ws, bytes, stream);
    });
  });
}

// (address of the cache, its pool, layer, q, cu_q, seq_lens, max_seq_len, out, workspace,
//  scale, stream or None)
PyObject* raw_cross(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const auto* cache = static_cast<const kvtc_raw_cache*>(address(a[0]));
    const at::Tensor& pool = tensor(a[1], "the cache");
    const int dev = device_of(pool, "the cache"), layer = small_integer(a[2], "layer");
    const at::Tensor& q = queries(a[3], pool, dev, -1);
    const auto* cu = static_cast<const int32_t*>(buffer(a[4], at::kInt, "cu_q", dev, cache->n_seq + 1ll));
    const auto* lens = static_cast<const int32_t*>(buffer(a[5], at::kInt, "seq_lens", dev, cache->n_seq));
    const int max_len = small_integer(a[6], "max_seq_len");
    void* out = buffer_like(a[7], q, "out", dev);
    uint64_t bytes = 0;
    void* ws = workspace(a[8], dev, bytes);
    const float scale = static_cast<float>(number(a[9]));
    void* stream = stream_of(a[10], dev);
    const int heads = count(q.size(1), "q"), tokens = count(q.size(0), "q");
    const void* qp = q.data_ptr();
    return without_gil([&] {
      return fns.raw_cross(cache, layer, qp, heads, cu, tokens, lens, max_len, scale, out, ws, bytes, stream);
    });
  });
}

// Addresses of the library's five functions, in the order of `fns`.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    fns.step_tables = reinterpret_cast<decltype(fns.step_tables)>(address(a[0]));
    fns.rope = reinterpret_cast<decltype(fns.rope)>(address(a[1]));
    fns.raw_append = reinterpret_cast<decltype(fns.raw_append)>(address(a[2]));
    fns.raw_decode = reinterpret_cast<decltype(fns.raw_decode)>(address(a[3]));
    fns.raw_cross = reinterpret_cast<decltype(fns.raw_cross)>(address(a[4]));
    return 0;
  });
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"step_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(step_tables)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope)), METH_FASTCALL, nullptr},
    {"raw_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(raw_append)), METH_FASTCALL, nullptr},
    {"raw_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(raw_decode)), METH_FASTCALL, nullptr},
    {"raw_cross", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(raw_cross)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
