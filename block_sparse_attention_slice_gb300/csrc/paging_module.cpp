// The marshalling of paging.py and beam.py in C++: checks tensors, allocates outputs
// and workspaces, and calls the C ABI of include/attn_paged.h and attn_beam.h on the tensors'
// device and the given or current stream.  A call of the paged attention runs
// for 10 us on the GPU at its smallest; the same marshalling in Python took 25.
// Nothing is kept from one call to the next.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <string>
#include <vector>

#include "../../include/attn_beam.h"
#include "../../include/attn_paged.h"

namespace {

using at::Tensor;

PyObject *g_error = nullptr;      // AttnError(code, where)

struct Raised {};                 // a Python error is set

[[noreturn]] void refuse(const std::string &why, PyObject *type = PyExc_ValueError) {
  PyErr_SetString(type, why.c_str());
  throw Raised();
}

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor", PyExc_TypeError);
  return THPVariable_Unpack(o);
}
const Tensor *maybe(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

int integer(PyObject *o, const char *name) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised();
  if (x > INT_MAX || x < INT_MIN) refuse(std::string(name) + " is out of range");
  return static_cast<int>(x);
}
int narrow(int64_t x, const char *name) {
  if (x > INT_MAX) refuse(std::string(name) + " is out of range");
  return static_cast<int>(x);
}

// An int32 vector on `device`, contiguous.
const int32_t *ints(const Tensor *t, const char *name, at::Device device) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->dim() != 1 || t->device() != device || !t->is_contiguous())
    refuse(std::string(name) + " must be a contiguous int32 vector on " + device.str());
  return static_cast<const int32_t *>(t->data_ptr());
}

// Pages of either kind: with scales they hold 8 bits a value.
struct PagesArg {
  attn_pages8_t p8;
  bool is8;
  const attn_pages_t &pages() const { return p8.pages; }
};
PagesArg pages_of(PyObject *ko, PyObject *vo, PyObject *kso, PyObject *vso) {
  const Tensor &k = tensor(ko, "k_pages"), &v = tensor(vo, "v_pages");
  const Tensor *ks = maybe(kso, "k_scales"), *vs = maybe(vso, "v_scales");
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.strides() != v.strides() || k.stride(3) != 1)
    refuse("k_pages and v_pages must be [n_pages, page_size, H_k, d], alike in strides, d contiguous");
  PagesArg a;
  a.is8 = ks || vs;
  const at::ScalarType want = a.is8 && k.scalar_type() == at::kChar ? at::kChar : a.is8 ? at::kFloat8_e4m3fn : at::kBFloat16;
  if (k.scalar_type() != want || v.scalar_type() != want || !k.is_cuda() || v.device() != k.device())
    refuse("k_pages and v_pages must be bf16 tensors, or int8 or float8_e4m3fn ones with k_scales and v_scales, on one CUDA device");
  if (a.is8) {
    if (!ks || !vs) refuse("k_scales and v_scales must be given together");
    if (ks->dim() != 3 || ks->sizes() != k.sizes().slice(0, 3) || vs->sizes() != ks->sizes() || vs->strides() != ks->strides() ||
        ks->scalar_type() != at::kFloat || vs->scalar_type() != at::kFloat || ks->device() != k.device() || vs->device() != k.device())
      refuse("k_scales and v_scales must be f32 [n_pages, page_size, H_k] on the pages' device, alike in strides");
    a.p8.k_scales = static_cast<const float *>(ks->data_ptr());
    a.p8.v_scales = static_cast<const float *>(vs->data_ptr());
    a.p8.scale_page_stride = ks->stride(0);
    a.p8.scale_token_stride = ks->stride(1);
    a.p8.scale_head_stride = ks->stride(2);
    a.p8.format = want == at::kChar ? ATTN_CODES_INT8 : ATTN_CODES_E4M3;
    a.p8.reserved = 0;
  }
  attn_pages_t &p = a.p8.pages;
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  p.n_pages = narrow(k.size(0), "n_pages");
  p.page_size = narrow(k.size(1), "page_size");
  p.hk = narrow(k.size(2), "H_k");
  p.d = narrow(k.size(3), "d");
  p.page_stride = k.stride(0);
  p.token_stride = k.stride(1);
  p.head_stride = k.stride(2);
  return a;
}

void check_rows(const Tensor &table, const Tensor &lens, at::Device device, const char *what) {
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.device() != device ||
      (table.size(1) > 1 && table.stride(1) != 1))
    refuse(std::string(what) + "table must be int32 [n_slots, max_pages] on " + device.str() + ", rows contiguous");
  ints(&lens, (std::string(what) + "seq_lens").c_str(), device);
  if (lens.size(0) != table.size(0)) refuse(std::string(what) + "table and its lengths must have one row a slot");
}
int64_t row_stride(const Tensor &table) {
  return table.size(0) > 1 ? table.stride(0) : std::max(table.size(1), table.stride(0));
}

attn_seqs_t seqs_of(PyObject *to, PyObject *lo, const Tensor *seqs, at::Device device, const char *what) {
  const Tensor &table = tensor(to, "table"), &lens = tensor(lo, "seq_lens");
  check_rows(table, lens, device, what);
  attn_seqs_t s;
  s.table = static_cast<const int32_t *>(table.data_ptr());
  s.seq_lens = static_cast<const int32_t *>(lens.data_ptr());
  s.seqs = ints(seqs, "seqs", device);
  s.table_stride = row_stride(table);
  s.n_slots = narrow(table.size(0), "n_slots");
  s.max_pages = narrow(table.size(1), "max_pages");
  s.n_seqs = seqs ? narrow(seqs->size(0), "n_seqs") : s.n_slots;
  s.reserved = 0;
  return s;
}

struct CacheArg {
  attn_cache_t c;
  at::Device device;
};
CacheArg cache_of(PyObject *to, PyObject *lo, PyObject *ro, PyObject *page) {
  const Tensor &table = tensor(to, "table"), &lens = tensor(lo, "seq_lens"), &refs = tensor(ro, "refs");
  if (!table.is_cuda()) refuse("the cache's arrays must be CUDA tensors");
  CacheArg a{{}, table.device()};
  check_rows(table, lens, a.device, "");
  a.c.table = static_cast<int32_t *>(table.data_ptr());
  a.c.seq_lens = static_cast<int32_t *>(lens.data_ptr());
  a.c.refs = const_cast<int32_t *>(ints(&refs, "refs", a.device));
  a.c.table_stride = row_stride(table);
  a.c.n_slots = narrow(table.size(0), "n_slots");
  a.c.max_pages = narrow(table.size(1), "max_pages");
  a.c.n_pages = narrow(refs.size(0), "n_pages");
  a.c.page_size = integer(page, "page_size");
  return a;
}

attn_stream_t stream_of(PyObject *o, at::Device device) {
  if (o == Py_None) return reinterpret_cast<attn_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised();
  return static_cast<attn_stream_t>(p);
}

// Calls f() on `device`, without the interpreter's lock (f neither throws nor
// refuses), and raises its error.
template <typename F>
void call(const char *name, at::Device device, F f) {
  int code;
  {
    c10::cuda::CUDAGuard guard(device);
    PyThreadState *save = PyEval_SaveThread();
    code = f();
    PyEval_RestoreThread(save);
  }
  if (code == ATTN_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", code, name);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

// Every entry: `n` positional arguments; C++ errors become Python's.
template <int N, PyObject *(*F)(PyObject *const *)>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Raised &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ error");
  }
  return nullptr;
}

// What both attention calls share.
struct Attend {
  const Tensor *q;
  const int32_t *q_ptr;
  int t, hq, max_q, out_dtype;
  float scale;
  Tensor out, lse, ws;
  PyObject *out_o, *lse_o;      // the caller's own, or null

  Attend(at::Device device, const attn_pages_t &pages, int n_seqs, PyObject *qo, PyObject *scale_o, PyObject *ptr_o,
         PyObject *max_o, PyObject *oo, PyObject *lo, PyObject *dt, PyObject *wo, int prefix) {
    q = &tensor(qo, "q");
    if (q->scalar_type() != at::kBFloat16 || q->dim() != 3 || q->device() != device || !q->is_contiguous())
      refuse("q must be a contiguous bf16 [n_tokens, H, d] tensor on " + device.str());
    if (q->size(2) != pages.d) refuse("q and the pages must have one head dim");
    t = narrow(q->size(0), "n_tokens");
    hq = narrow(q->size(1), "H");
    const Tensor *ptr = maybe(ptr_o, "q_ptr");
    q_ptr = ints(ptr, "q_ptr", device);
    if (ptr && ptr->size(0) != static_cast<int64_t>(n_seqs) + 1) refuse("q_ptr must have one entry a sequence and one more");
    scale = static_cast<float>(PyFloat_AsDouble(scale_o));
    if (PyErr_Occurred()) throw Raised();
    max_q = max_o != Py_None ? integer(max_o, "max_q") : ptr ? std::max(1, t) : 1;
    at::ScalarType want = at::kBFloat16;
    if (dt != Py_None) {
      if (!THPDtype_Check(dt)) refuse("out_dtype must be a dtype", PyExc_TypeError);
      want = reinterpret_cast<THPDtype *>(dt)->scalar_type;
    }
    out_o = oo == Py_None ? nullptr : oo;
    lse_o = lo == Py_None ? nullptr : lo;
    if (out_o) {
      out = tensor(oo, "out");
      if (out.sizes() != q->sizes() || out.device() != device || !out.is_contiguous() || (dt != Py_None && out.scalar_type() != want))
        refuse("out must be a contiguous bf16 or f32 tensor like q");
      want = out.scalar_type();
    }
    if (want != at::kBFloat16 && want != at::kFloat) refuse("out must be bf16 or f32");
    out_dtype = want == at::kFloat ? ATTN_DTYPE_F32 : ATTN_DTYPE_BF16;
    const auto on = at::TensorOptions().device(device);
    if (!out_o) out = at::empty(q->sizes(), on.dtype(want));
    if (lse_o) {
      lse = tensor(lo, "lse");
      if (lse.dim() != 2 || lse.size(0) != hq || lse.size(1) != t || lse.scalar_type() != at::kFloat || lse.device() != device ||
          !lse.is_contiguous())
        refuse("lse must be a contiguous f32 [H, n_tokens] tensor");
    } else {
      lse = at::empty({hq, t}, on.dtype(at::kFloat));
    }
    if (wo != Py_None) {
      ws = tensor(wo, "ws");
      if (ws.device() != device || !ws.is_contiguous()) refuse("ws must be a contiguous tensor on the queries' device");
    } else {
      size_t bytes = 0;
      call("attn_paged_workspace_bytes", device, [&] { return attn_paged_workspace_bytes(t, hq, pages.d, prefix, &bytes); });
      ws = at::empty({static_cast<int64_t>(bytes)}, on.dtype(at::kByte));
    }
  }
  size_t ws_bytes() const { return ws.nbytes(); }
  PyObject *result() const {
    PyObject *o = out_o ? Py_NewRef(out_o) : THPVariable_Wrap(out), *l = lse_o ? Py_NewRef(lse_o) : THPVariable_Wrap(lse);
    PyObject *r = o && l ? PyTuple_Pack(2, o, l) : nullptr;
    Py_XDECREF(o);
    Py_XDECREF(l);
    return r;
  }
};

// q, k_pages, v_pages, table, seq_lens, scale, q_ptr, max_q, window, sinks, seqs, out, lse, out_dtype, ws, stream, k_scales, v_scales
PyObject *paged_fwd(PyObject *const *a) {
  const PagesArg of = pages_of(a[1], a[2], a[16], a[17]);
  const attn_pages_t &pages = of.pages();
  const at::Device device = THPVariable_Unpack(a[1]).device();
  const attn_seqs_t seqs = seqs_of(a[3], a[4], maybe(a[10], "seqs"), device, "");
  const int window = integer(a[8], "window"), sinks = integer(a[9], "sinks");
  Attend x(device, pages, seqs.n_seqs, a[0], a[5], a[6], a[7], a[11], a[12], a[13], a[14], 0);
  attn_stream_t s = stream_of(a[15], device);
  if (of.is8)
    call("attn_paged8_fwd", device, [&] {
      return attn_paged8_fwd(x.q->data_ptr(), x.q_ptr, x.t, x.max_q, x.hq, &of.p8, &seqs, x.scale, window, sinks, x.out.data_ptr(),
                             x.out_dtype, static_cast<float *>(x.lse.data_ptr()), x.ws.data_ptr(), x.ws_bytes(), s);
    });
  else call("attn_paged_fwd", device, [&] {
    return attn_paged_fwd(x.q->data_ptr(), x.q_ptr, x.t, x.max_q, x.hq, &pages, &seqs, x.scale, window, sinks, x.out.data_ptr(),
                          x.out_dtype, static_cast<float *>(x.lse.data_ptr()), x.ws.data_ptr(), x.ws_bytes(), s);
  });
  return x.result();
}

// q, k_pages, v_pages, prefix_table, prefix_lens, group_ptr, table, seq_lens, scale, q_ptr, max_q, seqs, out, lse, out_dtype, ws, stream,
// k_scales, v_scales
PyObject *prefix_fwd(PyObject *const *a) {
  const PagesArg of = pages_of(a[1], a[2], a[17], a[18]);
  const attn_pages_t &pages = of.pages();
  const at::Device device = THPVariable_Unpack(a[1]).device();
  const attn_seqs_t pre = seqs_of(a[3], a[4], nullptr, device, "prefix_");
  const attn_seqs_t seqs = seqs_of(a[6], a[7], maybe(a[11], "seqs"), device, "");
  const Tensor &group = tensor(a[5], "group_ptr");
  const int32_t *group_ptr = ints(&group, "group_ptr", device);
  if (group.size(0) != static_cast<int64_t>(pre.n_seqs) + 1) refuse("group_ptr must have one entry a prefix and one more");
  Attend x(device, pages, seqs.n_seqs, a[0], a[8], a[9], a[10], a[12], a[13], a[14], a[15], 1);
  attn_stream_t s = stream_of(a[16], device);
  if (of.is8)
    call("attn_prefix8_fwd", device, [&] {
      return attn_prefix8_fwd(x.q->data_ptr(), x.q_ptr, x.t, x.max_q, x.hq, &of.p8, &pre, group_ptr, &seqs, x.scale, x.out.data_ptr(),
                              x.out_dtype, static_cast<float *>(x.lse.data_ptr()), x.ws.data_ptr(), x.ws_bytes(), s);
    });
  else call("attn_prefix_fwd", device, [&] {
    return attn_prefix_fwd(x.q->data_ptr(), x.q_ptr, x.t, x.max_q, x.hq, &pages, &pre, group_ptr, &seqs, x.scale, x.out.data_ptr(),
                           x.out_dtype, static_cast<float *>(x.lse.data_ptr()), x.ws.data_ptr(), x.ws_bytes(), s);
  });
  return x.result();
}

// table, seq_lens, refs, seqs, counts, page_size, stream
PyObject *cache_extend(PyObject *const *a) {
  const CacheArg c = cache_of(a[0], a[1], a[2], a[5]);
  const Tensor &seqs = tensor(a[3], "seqs"), &counts = tensor(a[4], "counts");
  const int32_t *s = ints(&seqs, "seqs", c.device), *add = ints(&counts, "counts", c.device);
  if (seqs.size(0) != counts.size(0)) refuse("seqs and counts must be of one length");
  const int n = narrow(seqs.size(0), "n");
  attn_stream_t st = stream_of(a[6], c.device);
  call("attn_cache_extend", c.device, [&] { return attn_cache_extend(&c.c, s, add, n, st); });
  Py_RETURN_NONE;
}

// table, seq_lens, refs, seqs, page_size, stream
PyObject *cache_free(PyObject *const *a) {
  const CacheArg c = cache_of(a[0], a[1], a[2], a[4]);
  const Tensor &seqs = tensor(a[3], "seqs");
  const int32_t *s = ints(&seqs, "seqs", c.device);
  const int n = narrow(seqs.size(0), "n");
  attn_stream_t st = stream_of(a[5], c.device);
  call("attn_cache_free", c.device, [&] { return attn_cache_free(&c.c, s, n, st); });
  Py_RETURN_NONE;
}

// table, seq_lens, refs, page_size, window, sinks, seqs, stream
PyObject *cache_trim(PyObject *const *a) {
  const CacheArg c = cache_of(a[0], a[1], a[2], a[3]);
  const int window = integer(a[4], "window"), sinks = integer(a[5], "sinks");
  const Tensor *seqs = maybe(a[6], "seqs");
  const int32_t *s = ints(seqs, "seqs", c.device);
  if (seqs && !s) s = c.c.seq_lens;      // a list of no rows has no address; to the call a null one is all rows
  const int n = seqs ? narrow(seqs->size(0), "n") : c.c.n_slots;
  attn_stream_t st = stream_of(a[7], c.device);
  call("attn_cache_trim", c.device, [&] { return attn_cache_trim(&c.c, s, n, window, sinks, st); });
  Py_RETURN_NONE;
}

// The copy list and the workspace of a call that makes one; either may be the caller's.
struct Copies {
  Tensor list, ws;
  int cap;
  Copies(const CacheArg &c, int64_t cap_, int n, PyObject *lo, PyObject *wo) : cap(narrow(cap_, "n")) {
    const auto on = at::TensorOptions().device(c.device);
    size_t bytes = 0;
    call("attn_cache_workspace_bytes", c.device, [&] { return attn_cache_workspace_bytes(&c.c, n, &bytes); });
    list = lo == Py_None ? at::empty({1 + 2 * static_cast<int64_t>(cap)}, on.dtype(at::kInt)) : tensor(lo, "copies");
    ws = wo == Py_None ? at::empty({static_cast<int64_t>(bytes)}, on.dtype(at::kByte)) : tensor(wo, "ws");
    ints(&list, "copies", c.device);
    if (list.size(0) != 1 + 2 * static_cast<int64_t>(cap)) refuse("copies must have 1 + 2 cap entries");
    if (ws.device() != c.device || !ws.is_contiguous()) refuse("ws must be a contiguous tensor on the cache's device");
  }
  int32_t *at() const { return static_cast<int32_t *>(list.data_ptr()); }
};

// table, seq_lens, refs, src, dst, page_size, copies, ws, stream
PyObject *cache_fork(PyObject *const *a) {
  const CacheArg c = cache_of(a[0], a[1], a[2], a[5]);
  const Tensor &src = tensor(a[3], "src"), &dst = tensor(a[4], "dst");
  const int32_t *s = ints(&src, "src", c.device), *d = ints(&dst, "dst", c.device);
  if (src.size(0) != dst.size(0)) refuse("src and dst must be of one length");
  const int n = narrow(src.size(0), "n");
  Copies x(c, n, n, a[6], a[7]);
  attn_stream_t st = stream_of(a[8], c.device);
  call("attn_cache_fork", c.device,
       [&] { return attn_cache_fork(&c.c, s, d, n, x.at(), x.cap, x.ws.data_ptr(), x.ws.nbytes(), st); });
  return a[6] == Py_None ? THPVariable_Wrap(x.list) : Py_NewRef(a[6]);
}

// table, seq_lens, refs, page_size, copies, ws, stream
PyObject *cache_compact(PyObject *const *a) {
  const CacheArg c = cache_of(a[0], a[1], a[2], a[3]);
  Copies x(c, c.c.n_pages / 2, 0, a[4], a[5]);
  attn_stream_t st = stream_of(a[6], c.device);
  call("attn_cache_compact", c.device,
       [&] { return attn_cache_compact(&c.c, x.at(), x.cap, x.ws.data_ptr(), x.ws.nbytes(), st); });
  return a[4] == Py_None ? THPVariable_Wrap(x.list) : Py_NewRef(a[4]);
}

// pools, copies, stream
PyObject *cache_copy_pages(PyObject *const *a) {
  PyObject *seq = PySequence_Fast(a[0], "pools must be a sequence of tensors");
  if (!seq) throw Raised();
  struct Drop {
    PyObject *o;
    ~Drop() { Py_DECREF(o); }
  } drop{seq};
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  if (n == 0) Py_RETURN_NONE;
  const Tensor &x = tensor(PySequence_Fast_GET_ITEM(seq, 0), "a pool");
  bool whole = x.is_cuda() && x.dim() >= 2 && x.size(0) > 0;
  int64_t run = 1;
  for (int64_t i = x.dim() - 1; whole && i >= 1; --i) {
    if (x.size(i) != 1 && x.stride(i) != run) whole = false;
    run *= x.size(i);
  }
  if (!whole) refuse("pools must be CUDA tensors [n_pages, ...], each page contiguous");
  std::vector<void *> at;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor &y = tensor(PySequence_Fast_GET_ITEM(seq, i), "a pool");
    if (y.sizes() != x.sizes() || y.strides() != x.strides() || y.element_size() != x.element_size() || y.device() != x.device())
      refuse("pools must be alike in shape, strides and element size, on one device");
    at.push_back(y.data_ptr());
  }
  const Tensor &list = tensor(a[1], "copies");
  const int32_t *copies = ints(&list, "copies", x.device());
  if (list.size(0) % 2 != 1) refuse("copies must be int32 [1 + 2 cap]");
  const size_t page = static_cast<size_t>(run) * x.element_size();
  const size_t stride = x.size(0) > 1 ? static_cast<size_t>(x.stride(0)) * x.element_size() : page;
  const int n_pages = narrow(x.size(0), "n_pages"), cap = narrow(list.size(0) / 2, "cap");
  attn_stream_t st = stream_of(a[2], x.device());
  call("attn_cache_copy_pages", x.device(), [&] {
    return attn_cache_copy_pages(at.data(), static_cast<int>(n > INT_MAX ? INT_MAX : n), page, stride, n_pages, copies, cap, st);
  });
  Py_RETURN_NONE;
}

// k_pages, v_pages, k_new, v_new, table, seq_lens, q_ptr, seqs, stream, k_scales, v_scales
PyObject *cache_write(PyObject *const *a) {
  const PagesArg of = pages_of(a[0], a[1], a[9], a[10]);
  const attn_pages_t &pages = of.pages();
  const at::Device device = THPVariable_Unpack(a[0]).device();
  const attn_seqs_t seqs = seqs_of(a[4], a[5], maybe(a[7], "seqs"), device, "");
  const Tensor *ptr = maybe(a[6], "q_ptr");
  const int32_t *q_ptr = ints(ptr, "q_ptr", device);
  if (ptr && ptr->size(0) != static_cast<int64_t>(seqs.n_seqs) + 1) refuse("q_ptr must have one entry a sequence and one more");
  const Tensor &k = tensor(a[2], "k_new"), &v = tensor(a[3], "v_new");
  if (k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16 || k.device() != device || v.device() != device ||
      k.dim() != 3 || k.sizes() != v.sizes() || k.size(1) != pages.hk || k.size(2) != pages.d || k.strides() != v.strides() ||
      k.stride(2) != 1)
    refuse("k_new and v_new must be bf16 [n_tokens, H_k, d] on the pages' device, alike in strides, d contiguous");
  const int t = narrow(k.size(0), "n_tokens");
  attn_stream_t st = stream_of(a[8], device);
  if (of.is8)
    call("attn_cache8_write", device,
         [&] { return attn_cache8_write(&of.p8, &seqs, q_ptr, k.data_ptr(), v.data_ptr(), t, k.stride(0), k.stride(1), st); });
  else
    call("attn_cache_write", device,
         [&] { return attn_cache_write(&pages, &seqs, q_ptr, k.data_ptr(), v.data_ptr(), t, k.stride(0), k.stride(1), st); });
  Py_RETURN_NONE;
}

// k_pages, v_pages, table, seq_lens, n_tokens, q_ptr, seqs, k_out, v_out, out_dtype, stream, k_scales, v_scales
PyObject *cache_read(PyObject *const *a) {
  const PagesArg of = pages_of(a[0], a[1], a[11], a[12]);
  const attn_pages_t &pages = of.pages();
  const at::Device device = THPVariable_Unpack(a[0]).device();
  const attn_seqs_t seqs = seqs_of(a[2], a[3], maybe(a[6], "seqs"), device, "");
  const int t = integer(a[4], "n_tokens");
  if (t < 0) refuse("n_tokens must not be negative");
  const Tensor *ptr = maybe(a[5], "q_ptr");
  const int32_t *q_ptr = ints(ptr, "q_ptr", device);
  if (ptr && ptr->size(0) != static_cast<int64_t>(seqs.n_seqs) + 1) refuse("q_ptr must have one entry a sequence and one more");
  at::ScalarType want = at::kBFloat16;
  if (a[9] != Py_None) {
    if (!THPDtype_Check(a[9])) refuse("out_dtype must be a dtype", PyExc_TypeError);
    want = reinterpret_cast<THPDtype *>(a[9])->scalar_type;
  }
  if ((a[7] == Py_None) != (a[8] == Py_None)) refuse("k_out and v_out must be given together");
  const std::vector<int64_t> sizes{t, pages.hk, pages.d};
  Tensor out[2];
  for (int i = 0; i < 2; ++i) {
    PyObject *o = a[7 + i];
    if (o == Py_None) continue;
    out[i] = tensor(o, i ? "v_out" : "k_out");
    if (out[i].sizes() != at::IntArrayRef(sizes) || out[i].device() != device || !out[i].is_contiguous() ||
        (a[9] != Py_None && out[i].scalar_type() != want) || out[i].scalar_type() != out[0].scalar_type())
      refuse("k_out and v_out must be contiguous bf16 or f32 [n_tokens, H_k, d] tensors, of one type, on the pages' device");
    if (i == 0) want = out[0].scalar_type();
  }
  if (want != at::kBFloat16 && want != at::kFloat) refuse("the rows must be bf16 or f32");
  if (a[7] == Py_None)
    for (Tensor &x : out) x = at::empty(sizes, at::TensorOptions().device(device).dtype(want));
  const int dtype = want == at::kFloat ? ATTN_DTYPE_F32 : ATTN_DTYPE_BF16;
  attn_stream_t st = stream_of(a[10], device);
  if (of.is8)
    call("attn_cache8_read", device,
         [&] { return attn_cache8_read(&of.p8, &seqs, q_ptr, t, out[0].data_ptr(), out[1].data_ptr(), dtype, st); });
  else
    call("attn_cache_read", device,
         [&] { return attn_cache_read(&pages, &seqs, q_ptr, t, out[0].data_ptr(), out[1].data_ptr(), dtype, st); });
  PyObject *k = a[7] == Py_None ? THPVariable_Wrap(out[0]) : Py_NewRef(a[7]), *v = a[8] == Py_None ? THPVariable_Wrap(out[1]) : Py_NewRef(a[8]);
  PyObject *r = k && v ? PyTuple_Pack(2, k, v) : nullptr;
  Py_XDECREF(k);
  Py_XDECREF(v);
  return r;
}

// logits, scores, done, eos, slots, keep, ws, stream
PyObject *beam_select(PyObject *const *a) {
  const Tensor &logits = tensor(a[0], "logits"), &scores = tensor(a[1], "scores");
  const Tensor *done = maybe(a[2], "done"), *slots = maybe(a[4], "slots");
  if (!logits.is_cuda() || (logits.scalar_type() != at::kFloat && logits.scalar_type() != at::kBFloat16) || logits.dim() != 2 ||
      (logits.stride(1) != 1 && logits.size(1) != 1))
    refuse("logits must be f32 or bf16 [groups * beams, vocab] on a CUDA device, rows contiguous");
  const at::Device device = logits.device();
  if (scores.scalar_type() != at::kFloat || scores.dim() != 2 || scores.device() != device || !scores.is_contiguous())
    refuse("scores must be a contiguous f32 [groups, beams] tensor on " + device.str());
  const int groups = narrow(scores.size(0), "groups"), beams = narrow(scores.size(1), "beams"), vocab = narrow(logits.size(1), "vocab");
  if (logits.size(0) != static_cast<int64_t>(groups) * beams) refuse("logits must have one row a beam");
  if (done && ((done->scalar_type() != at::kBool && done->scalar_type() != at::kByte) || done->sizes() != scores.sizes() || done->device() != device ||
               !done->is_contiguous()))
    refuse("done must be a contiguous bool or uint8 tensor like scores");
  const int32_t *slot = ints(slots, "slots", device);
  if (slots && slots->size(0) != logits.size(0)) refuse("slots must have one entry a beam");
  const int eos = integer(a[3], "eos"), keep = a[5] == Py_None ? beams : integer(a[5], "keep");
  size_t bytes = 0;
  call("attn_beam_workspace_bytes", device, [&] { return attn_beam_workspace_bytes(groups, beams, vocab, keep, &bytes); });
  const auto on = at::TensorOptions().device(device);
  Tensor ws = a[6] == Py_None ? at::empty({static_cast<int64_t>(bytes)}, on.dtype(at::kByte)) : tensor(a[6], "ws");
  if (ws.device() != device || !ws.is_contiguous()) refuse("ws must be a contiguous tensor on the logits' device");
  Tensor out[5];
  const at::ScalarType types[5] = {at::kFloat, at::kInt, at::kInt, at::kBool, at::kInt};
  const int n = slots ? 5 : 4;
  for (int i = 0; i < n; ++i) out[i] = at::empty({groups, keep}, on.dtype(types[i]));
  attn_stream_t st = stream_of(a[7], device);
  const int64_t stride = logits.size(0) > 1 ? logits.stride(0) : std::max<int64_t>(vocab, logits.stride(0));
  call("attn_beam_select", device, [&] {
    return attn_beam_select(logits.data_ptr(), logits.scalar_type() == at::kFloat ? ATTN_DTYPE_F32 : ATTN_DTYPE_BF16, stride, groups, beams, vocab,
                            static_cast<const float *>(scores.data_ptr()), done ? static_cast<const uint8_t *>(done->data_ptr()) : nullptr, eos, slot,
                            keep, static_cast<float *>(out[0].data_ptr()), static_cast<int32_t *>(out[1].data_ptr()),
                            static_cast<int32_t *>(out[2].data_ptr()), static_cast<uint8_t *>(out[3].data_ptr()),
                            slots ? static_cast<int32_t *>(out[4].data_ptr()) : nullptr, ws.data_ptr(), ws.nbytes(), st);
  });
  PyObject *r = PyTuple_New(n);
  for (int i = 0; r && i < n; ++i) {
    PyObject *o = THPVariable_Wrap(out[i]);
    if (!o) Py_CLEAR(r);
    else PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// states, parents, stream
PyObject *beam_reorder(PyObject *const *a) {
  const Tensor &parents = tensor(a[1], "parents");
  if (parents.scalar_type() != at::kInt || parents.dim() != 2 || !parents.is_cuda() || !parents.is_contiguous())
    refuse("parents must be a contiguous int32 [groups, beams] CUDA tensor");
  const at::Device device = parents.device();
  PyObject *seq = PySequence_Fast(a[0], "states must be a sequence of tensors");
  if (!seq) throw Raised();
  struct Drop {
    PyObject *o;
    ~Drop() { Py_DECREF(o); }
  } drop{seq};
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  std::vector<void *> at;
  std::vector<int64_t> bytes, strides;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor &x = tensor(PySequence_Fast_GET_ITEM(seq, i), "a state");
    bool whole = x.device() == device && x.dim() >= 1 && x.size(0) == parents.numel();
    int64_t run = 1;
    for (int64_t k = x.dim() - 1; whole && k >= 1; --k) {
      if (x.size(k) != 1 && x.stride(k) != run) whole = false;
      run *= x.size(k);
    }
    if (!whole) refuse("states must be [groups * beams, ...] on " + device.str() + ", each row contiguous");
    at.push_back(x.data_ptr());
    bytes.push_back(run * static_cast<int64_t>(x.element_size()));
    strides.push_back(x.size(0) > 1 ? x.stride(0) * static_cast<int64_t>(x.element_size()) : bytes.back());
  }
  const int groups = narrow(parents.size(0), "groups"), beams = narrow(parents.size(1), "beams");
  attn_stream_t st = stream_of(a[2], device);
  call("attn_beam_reorder", device, [&] {
    return attn_beam_reorder(at.data(), bytes.data(), strides.data(), static_cast<int>(n > INT_MAX ? INT_MAX : n),
                             static_cast<const int32_t *>(parents.data_ptr()), groups, beams, st);
  });
  Py_RETURN_NONE;
}

PyObject *set_error(PyObject *, PyObject *cls) {
  Py_XSETREF(g_error, Py_NewRef(cls));
  Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<n, name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(paged_fwd, 18),   ENTRY(prefix_fwd, 19), ENTRY(cache_extend, 7), ENTRY(cache_free, 6),        ENTRY(cache_trim, 8),
                         ENTRY(cache_fork, 9),   ENTRY(cache_compact, 7), ENTRY(cache_copy_pages, 3), ENTRY(cache_write, 11), ENTRY(cache_read, 13),
                         ENTRY(beam_select, 8),  ENTRY(beam_reorder, 3), {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paging", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paging() { return PyModule_Create(&module); }
