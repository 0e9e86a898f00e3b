// Argument marshalling of the entry points that serve small, frequent calls
// (drafted trees, windows, pages), compiled: a call from Python costs its checks,
// output allocations and the launch, and in interpreted code the first two took
// two thirds of its 20 to 25 us.  binding.py's functions of the same names parse
// and document the arguments, bring the right device and stream to the fore and
// call these with all of them in order; a function here returns its results, or
// the entry point's status where that is not WF_OK.
//
// Only torch supplies device memory and the current stream; everything else is
// the C ABI (wavefilter.h).  No exception leaves a function: a bad argument
// becomes ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <sstream>
#include <stdexcept>
#include <string>

#include "wavefilter.h"

namespace {

struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void bad(const char* name, const std::string& want, const at::Tensor* got = nullptr) {
  std::ostringstream s;
  s << name << " must be " << want;
  if (got != nullptr)
    s << ", got " << c10::toString(got->scalar_type()) << " " << got->sizes() << " on "
      << got->device() << ", strides " << got->strides();
  throw BadArgument(s.str());
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(name, "a tensor");
  return THPVariable_Unpack(o);
}

// A contiguous tensor of this type and shape on the device.
void* need(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type,
           const at::Device& dev) {
  if (t.scalar_type() != type || t.device() != dev || t.sizes() != shape || !t.is_contiguous()) {
    std::ostringstream s;
    s << "a contiguous " << c10::toString(type) << " tensor " << shape << " on " << dev;
    bad(name, s.str(), &t);
  }
  return t.data_ptr();
}
void* need(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type,
           const at::Device& dev) {
  return need(tensor(o, name), name, shape, type, dev);
}
int32_t* ints(PyObject* o, const char* name, at::IntArrayRef shape, const at::Device& dev) {
  return static_cast<int32_t*>(need(o, name, shape, at::kInt, dev));
}
int32_t* ints_or_none(PyObject* o, const char* name, at::IntArrayRef shape,
                      const at::Device& dev) {
  return o == Py_None ? nullptr : ints(o, name, shape, dev);
}

int dtype_of(at::ScalarType t) {
  if (t == at::kBFloat16) return WF_BF16;
  if (t == at::kFloat) return WF_F32;
  throw BadArgument(std::string("unsupported dtype ") + c10::toString(t));
}

int32_t size32(int64_t n, const char* name) {
  if (n < 0 || n > INT32_MAX) bad(name, "a size of 32 bits");
  return static_cast<int32_t>(n);
}
int32_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(name, "a whole number");
  }
  if (v < INT32_MIN || v > INT32_MAX) bad(name, "a number of 32 bits");
  return static_cast<int32_t>(v);
}
double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(name, "a number");
  }
  return v;
}
bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    bad(name, "a truth value");
  }
  return v != 0;
}

// In the struct 0 stands for the defaults: what fp32 rounds to it is refused.
wf_attn_opts options(PyObject* causal, PyObject* softcap, PyObject* slopes, PyObject* scale,
                     int64_t q_heads, const at::Device& dev) {
  wf_attn_opts o = {};
  if (scale != Py_None) {
    o.scale = static_cast<float>(number(scale, "scale"));
    if (o.scale == 0.f)
      throw BadArgument("scale must not be 0 in fp32 (None means 1/sqrt(head_dim))");
  }
  const double cap = number(softcap, "softcap");
  o.softcap = static_cast<float>(cap);
  if (cap != 0.0 && o.softcap == 0.f)
    throw BadArgument("softcap must not round to 0 in fp32 (0 means none)");
  o.causal = truth(causal, "causal");
  if (slopes != Py_None)
    o.slopes = static_cast<const float*>(need(slopes, "slopes", {q_heads}, at::kFloat, dev));
  return o;
}

struct Workspace {
  void* at;
  size_t bytes;
};
Workspace workspace(PyObject* o, const at::Device& dev) {
  if (o == Py_None) return {nullptr, 0};
  const at::Tensor& t = tensor(o, "workspace");
  return {need(t, "workspace", {t.numel()}, at::kByte, dev), static_cast<size_t>(t.numel())};
}

void* stream_of(const at::Device& dev) {
  return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
}

at::Tensor result(PyObject* given, const char* name, at::IntArrayRef shape, at::ScalarType type,
                  const at::Device& dev) {
  if (given == Py_None) return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  const at::Tensor& t = tensor(given, name);
  need(t, name, shape, type, dev);
  return t;
}

// The results of an attention call.
PyObject* attention(int status, const at::Tensor& o, const at::Tensor& lse) {
  if (status != WF_OK) return PyLong_FromLong(status);
  if (!lse.defined()) return THPVariable_Wrap(o);
  PyObject* x = THPVariable_Wrap(o);
  PyObject* y = x == nullptr ? nullptr : THPVariable_Wrap(lse);
  PyObject* r = y == nullptr ? nullptr : PyTuple_Pack(2, x, y);
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// A paged attention's queries, cache and table.
struct Paged {
  wf_page_dims dims;
  at::Device dev;
  at::ScalarType type;
  int64_t n_seqs, n_new, q_heads, d;
  void *q, *k, *v;
  int32_t* table;
};
Paged paged(PyObject* q, PyObject* k, PyObject* v, PyObject* table) {
  const at::Tensor& tq = tensor(q, "q");
  const at::Tensor& tk = tensor(k, "cache K");
  const at::Tensor& tt = tensor(table, "page_table");
  if (tq.dim() != 4) bad("q", "[n_seqs, n_new, q_heads, head_dim]", &tq);
  if (tk.dim() != 4) bad("cache K", "[n_pages, kv_heads, page_size, head_dim]", &tk);
  if (tt.dim() != 2) bad("page_table", "[n_seqs, table_pages]", &tt);
  Paged p = {{}, tq.device(), tq.scalar_type(), tt.size(0), tq.size(1), tq.size(2), tk.size(3),
             nullptr, nullptr, nullptr, nullptr};
  p.dims.n_seqs = size32(p.n_seqs, "n_seqs");
  p.dims.q_heads = size32(p.q_heads, "q_heads");
  p.dims.kv_heads = size32(tk.size(1), "kv_heads");
  p.dims.head_dim = size32(p.d, "head_dim");
  p.dims.page_size = size32(tk.size(2), "page_size");
  p.dims.n_pages = size32(tk.size(0), "n_pages");
  p.dims.table_pages = size32(tt.size(1), "table_pages");
  p.dims.dtype = dtype_of(p.type);
  p.q = need(tq, "q", {p.n_seqs, p.n_new, p.q_heads, p.d}, p.type, p.dev);
  p.k = need(tk, "cache K", tk.sizes(), p.type, p.dev);
  p.v = need(v, "cache V", tk.sizes(), p.type, p.dev);
  p.table = ints(table, "page_table", tt.sizes(), p.dev);
  return p;
}

// q, K, V, page_table, kv_len, parents, ws, tree_len, softcap, slopes, scale, out, with_lse
PyObject* paged_tree(PyObject* const* a) {
  const Paged p = paged(a[0], a[1], a[2], a[3]);
  const wf_attn_opts o = options(Py_True, a[8], a[9], a[10], p.q_heads, p.dev);
  const int32_t* len = ints(a[4], "kv_len", {p.n_seqs}, p.dev);
  const int32_t* parents = ints(a[5], "parents", {p.n_seqs, p.n_new}, p.dev);
  const int32_t* count = ints_or_none(a[7], "tree_len", {p.n_seqs}, p.dev);
  const Workspace ws = workspace(a[6], p.dev);
  const at::Tensor out = result(a[11], "out", {p.n_seqs, p.n_new, p.q_heads, p.d}, p.type, p.dev);
  at::Tensor lse;
  if (truth(a[12], "with_lse"))
    lse = result(Py_None, "lse", {p.n_seqs, p.n_new, p.q_heads}, at::kFloat, p.dev);
  return attention(
      wf_paged_tree_attn(&p.dims, &o, size32(p.n_new, "n_nodes"), p.q, p.k, p.v, p.table, len,
                         parents, count, out.data_ptr(),
                         lse.defined() ? lse.data_ptr<float>() : nullptr, ws.at, ws.bytes,
                         stream_of(p.dev)),
      out, lse);
}

// q, K, V, page_table, kv_len, window, sinks, ws, causal, softcap, slopes, scale, out, with_lse
PyObject* paged_window(PyObject* const* a) {
  const Paged p = paged(a[0], a[1], a[2], a[3]);
  const wf_attn_opts o = options(a[8], a[9], a[10], a[11], p.q_heads, p.dev);
  const int32_t* len = ints(a[4], "kv_len", {p.n_seqs}, p.dev);
  const int32_t window = integer(a[5], "window"), sinks = integer(a[6], "sinks");
  const Workspace ws = workspace(a[7], p.dev);
  const at::Tensor out = result(a[12], "out", {p.n_seqs, p.n_new, p.q_heads, p.d}, p.type, p.dev);
  at::Tensor lse;
  if (truth(a[13], "with_lse"))
    lse = result(Py_None, "lse", {p.n_seqs, p.n_new, p.q_heads}, at::kFloat, p.dev);
  return attention(
      wf_paged_window_attn(&p.dims, &o, window, sinks, size32(p.n_new, "n_new"), p.q, p.k, p.v,
                           p.table, len, out.data_ptr(),
                           lse.defined() ? lse.data_ptr<float>() : nullptr, ws.at, ws.bytes,
                           stream_of(p.dev)),
      out, lse);
}

// Row stride of a [rows, heads, d] tensor whose rows may lie apart.
int64_t row_stride(const at::Tensor& t, const char* name, int64_t rows, int64_t heads, int64_t d,
                   at::ScalarType type, const at::Device& dev) {
  if (t.scalar_type() != type || t.device() != dev || t.dim() != 3 || t.size(0) != rows ||
      t.size(1) != heads || t.size(2) != d) {
    std::ostringstream s;
    s << "a " << c10::toString(type) << " tensor [" << rows << ", " << heads << ", " << d
      << "] on " << dev;
    bad(name, s.str(), &t);
  }
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
    bad(name, "rows of contiguous heads", &t);
  return rows > 1 ? t.stride(0) : heads * d;
}

// q, k, v, cu_q, cu_k, window, sinks, causal, softcap, slopes, scale, out, with_lse, ws
PyObject* prefill_window(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  if (q.dim() != 3) bad("q", "[rows, q_heads, head_dim]", &q);
  if (k.dim() != 3) bad("k", "[rows, kv_heads, head_dim]", &k);
  const at::Device dev = q.device();
  const at::ScalarType type = q.scalar_type();
  const int64_t t = q.size(0), hq = q.size(1), d = q.size(2), tk = k.size(0), hkv = k.size(1);
  const int64_t qs = row_stride(q, "q", t, hq, d, type, dev);
  const int64_t ks = row_stride(k, "k", tk, hkv, d, type, dev);
  const int64_t vs = row_stride(v, "v", tk, hkv, d, type, dev);
  const int64_t docs = tensor(a[3], "cu_q").numel() - 1;
  const int32_t* cq = ints(a[3], "cu_q", {docs + 1}, dev);
  const int32_t* ck = a[4] == Py_None ? cq : ints(a[4], "cu_k", {docs + 1}, dev);
  wf_prefill_dims dims = {size32(t, "rows_q"), size32(tk, "rows_k"), size32(docs, "n_docs"),
                          size32(hq, "q_heads"), size32(hkv, "kv_heads"),
                          size32(d, "head_dim"), dtype_of(type)};
  const wf_attn_opts o = options(a[7], a[8], a[9], a[10], hq, dev);
  const int32_t window = integer(a[5], "window"), sinks = integer(a[6], "sinks");
  const Workspace ws = workspace(a[13], dev);
  const at::Tensor out = result(a[11], "out", {t, hq, d}, type, dev);
  at::Tensor lse;
  if (truth(a[12], "with_lse")) lse = result(Py_None, "lse", {t, hq}, at::kFloat, dev);
  return attention(
      wf_prefill_window_attn(&dims, &o, window, sinks, q.data_ptr(), qs, k.data_ptr(), ks,
                             v.data_ptr(), vs, cq, ck, out.data_ptr(),
                             lse.defined() ? lse.data_ptr<float>() : nullptr, ws.at, ws.bytes,
                             stream_of(dev)),
      out, lse);
}

// A call on pages: one layer's pages (for the sizes), counts and table.
struct Pages {
  wf_page_dims dims;
  at::Device dev;
  int64_t n_seqs;
  int32_t *refs, *table;
};
Pages pages(PyObject* k, PyObject* refs, PyObject* table) {
  const at::Tensor& tk = tensor(k, "cache K");
  const at::Tensor& tt = tensor(table, "page_table");
  if (tk.dim() != 4) bad("cache K", "[n_pages, kv_heads, page_size, head_dim]", &tk);
  if (tt.dim() != 2) bad("page_table", "[n_seqs, table_pages]", &tt);
  Pages p = {{}, tk.device(), tt.size(0), nullptr, nullptr};
  p.dims.n_seqs = size32(tt.size(0), "n_seqs");
  p.dims.q_heads = p.dims.kv_heads = size32(tk.size(1), "kv_heads");
  p.dims.head_dim = size32(tk.size(3), "head_dim");
  p.dims.page_size = size32(tk.size(2), "page_size");
  p.dims.n_pages = size32(tk.size(0), "n_pages");
  p.dims.table_pages = size32(tt.size(1), "table_pages");
  p.dims.dtype = dtype_of(tk.scalar_type());
  p.table = ints(table, "page_table", tt.sizes(), p.dev);
  p.refs = ints_or_none(refs, "refs", {tk.size(0)}, p.dev);
  return p;
}
PyObject* status(int s) { return PyLong_FromLong(s); }

// The pointers of a pools handle: bytes of an array of addresses.
struct Pointers {
  void* const* at;
  int32_t n;
};
Pointers pointers(PyObject* o) {
  char* data = nullptr;
  Py_ssize_t bytes = 0;
  if (PyBytes_AsStringAndSize(o, &data, &bytes) != 0) {
    PyErr_Clear();
    bad("pools", "a handle's pointers");
  }
  return {reinterpret_cast<void* const*>(data), static_cast<int32_t>(bytes / sizeof(void*))};
}

// K, page_table, refs, rows, ws, from_rows
PyObject* reserve(PyObject* const* a) {
  const Pages p = pages(a[0], a[2], a[1]);
  const int32_t* rows = ints(a[3], "rows", {p.n_seqs}, p.dev);
  const Workspace ws = workspace(a[4], p.dev);
  const int32_t* from = ints_or_none(a[5], "from_rows", {p.n_seqs}, p.dev);
  return status(wf_paged_reserve_from(&p.dims, from, rows, p.refs, p.table, ws.at, ws.bytes,
                                      stream_of(p.dev)));
}

// pointers, K, page_table, refs, src, dst, kv_len, share_rows, ws
PyObject* fork(PyObject* const* a) {
  const Pointers pools = pointers(a[0]);
  const Pages p = pages(a[1], a[3], a[2]);
  const int64_t n = tensor(a[4], "src").numel();
  const int32_t* src = ints(a[4], "src", {n}, p.dev);
  const int32_t* dst = ints(a[5], "dst", {n}, p.dev);
  const int32_t* len = ints(a[6], "kv_len", {p.n_seqs}, p.dev);
  const int32_t* share = ints_or_none(a[7], "share_rows", {n}, p.dev);
  const Workspace ws = workspace(a[8], p.dev);
  return status(wf_paged_fork(&p.dims, size32(n, "n_forks"), src, dst, len, share, p.refs, p.table,
                              pools.n, pools.at, ws.at, ws.bytes, stream_of(p.dev)));
}

// pointers, K, page_table, refs, kv_len, start, keep, n_keep, ws
PyObject* keep(PyObject* const* a) {
  const Pointers pools = pointers(a[0]);
  const Pages p = pages(a[1], a[3], a[2]);
  const int32_t* len = ints(a[4], "kv_len", {p.n_seqs}, p.dev);
  const int32_t* start = ints(a[5], "start", {p.n_seqs}, p.dev);
  int64_t most = 0;
  if (a[6] != Py_None) {
    const at::Tensor& t = tensor(a[6], "keep");
    if (t.dim() != 2) bad("keep", "[n_seqs, max_keep]", &t);
    most = t.size(1);
  }
  const int32_t* rows = ints_or_none(a[6], "keep", {p.n_seqs, most}, p.dev);
  const int32_t* count = ints_or_none(a[7], "n_keep", {p.n_seqs}, p.dev);
  const Workspace ws = workspace(a[8], p.dev);
  return status(wf_paged_keep(&p.dims, len, start, rows, size32(most, "max_keep"), count, p.refs,
                              p.table, pools.n, pools.at, ws.at, ws.bytes, stream_of(p.dev)));
}

// K, page_table, refs, first, end, ws
PyObject* release(PyObject* const* a) {
  const Pages p = pages(a[0], a[2], a[1]);
  const int32_t* first = ints(a[3], "first", {p.n_seqs}, p.dev);
  const int32_t* end = ints(a[4], "end", {p.n_seqs}, p.dev);
  const Workspace ws = workspace(a[5], p.dev);
  return status(
      wf_paged_release(&p.dims, first, end, p.refs, p.table, ws.at, ws.bytes, stream_of(p.dev)));
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != N) throw BadArgument("wrong number of arguments");
    return F(args);
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {  // torch's own: out of memory and the like
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {method<paged_tree, 13>("paged_tree"),
                          method<paged_window, 14>("paged_window"),
                          method<prefill_window, 14>("prefill_window"),
                          method<reserve, 6>("reserve"),
                          method<fork, 9>("fork"),
                          method<keep, 9>("keep"),
                          method<release, 6>("release"),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_wf_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__wf_torch() { return PyModule_Create(&kModule); }
