// Python entry of the operators of include/gdn_block.h (the functions of block.py): argument checks, output and workspace
// tensors from PyTorch's allocator, the current stream, and the call of the C entry point.
//
// It is a C++ extension, not ctypes, because a decode step's operators take 3 to 10 us on the GPU: checking a dozen
// tensors, filling a shape struct and allocating outputs took 13 to 20 us of host time in Python.  The C entry points
// are called through addresses that the binding hands over once (connect), so the two libraries stay separate.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/gdn_block.h"

namespace {

using at::Tensor;

// ------------------------------------------------------------------ the C entry points
struct Api {
  decltype(&gdn_paged_attn_workspace_size) paged_attn_workspace_size;
  decltype(&gdn_paged_attn_fwd) paged_attn_fwd;
  decltype(&gdn_paged_attn_status) paged_attn_status;
  decltype(&gdn_rotary) rotary;
  decltype(&gdn_rotary_append) rotary_append;
  decltype(&gdn_slots_copy) slots_copy;
  decltype(&gdn_pages_workspace_size) pages_workspace_size;
  decltype(&gdn_pages_extend) pages_extend;
  decltype(&gdn_pages_fork) pages_fork;
  decltype(&gdn_pages_free) pages_free;
  decltype(&gdn_pages_compact) pages_compact;
  decltype(&gdn_rmsnorm_fwd) rmsnorm_fwd;
  decltype(&gdn_rmsnorm_bwd_workspace_size) rmsnorm_bwd_workspace_size;
  decltype(&gdn_rmsnorm_bwd) rmsnorm_bwd;
  decltype(&gdn_status_string) status_string;
  decltype(&gdn_last_error_string) last_error_string;
} api;
bool connected = false;

struct ValueError : std::runtime_error {
  using std::runtime_error::runtime_error;
};
[[noreturn]] void bad(const std::string &s) { throw ValueError(s); }
void check(int rc, const char *what) {
  if (rc) throw std::runtime_error(std::string(what) + ": " + api.status_string(rc) + " (" + api.last_error_string() + ")");
}

// ------------------------------------------------------------------ arguments
const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const Tensor *maybe(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }
int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::invalid_argument("");
  return v;
}
int small_int(PyObject *o, const char *name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + " does not fit 32 bits");
  return (int)v;
}
int fits(int64_t v, const char *name) {
  if (v > INT32_MAX) bad(std::string(name) + " is too large");
  return (int)v;
}
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw std::invalid_argument("");
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw std::invalid_argument("");
  return v;
}

// ------------------------------------------------------------------ checks
void here(const Tensor &t, const char *name) {
  if (!t.is_cuda() || t.get_device() != c10::cuda::current_device()) bad(std::string(name) + " must be on the current CUDA device");
}
void features(const Tensor &t, const char *name) {
  here(t, name);
  if (t.dim() < 1) bad(std::string(name) + " needs a feature dimension");
  if (t.size(-1) > 1 && t.stride(-1) != 1) bad(std::string("the last dimension of ") + name + " must be contiguous");
}
void heads(const Tensor &t, const char *name) {
  if (t.dim() != 3) bad(std::string(name) + " must have 3 dimensions [tokens, heads, features]");
  features(t, name);
}
// of a tensor that is written: no two of its elements may be one (an expanded dimension), or threads would race on it
void written(const Tensor &t, const char *name) {
  for (int64_t d = 0; d < t.dim(); ++d)
    if (t.size(d) > 1 && t.stride(d) == 0) bad(std::string(name) + " is written, so it must not be expanded");
}
void same_type(const Tensor &t, const Tensor &q, const char *name) {
  if (t.scalar_type() != q.scalar_type()) bad(std::string(name) + " must have the dtype of the other inputs");
}
void ints(const Tensor &t, const char *name) {
  if (t.scalar_type() != at::kInt) bad(std::string(name) + " must be an int32 tensor");
  here(t, name);
  if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
}
void ints(const Tensor &t, const char *name, int64_t n) {
  ints(t, name);
  if (t.dim() != 1 || t.size(0) != n) bad(std::string(name) + " must have " + std::to_string(n) + " entries");
}
gdn_dtype dtype(const Tensor &t, const char *name) {
  if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
  if (t.scalar_type() == at::kFloat) return GDN_FP32;
  bad(std::string(name) + " must be bfloat16 or float32");
}
void page_table(const Tensor &t) {
  if (t.dim() != 2 || t.scalar_type() != at::kInt || (t.size(1) > 1 && t.stride(1) != 1))
    bad("page_table must be an int32 CUDA tensor [sequences, pages] with contiguous rows");
  here(t, "page_table");
}
// of a table's rows, as it is (0 where one row is expanded over all sequences); one row alone may have any
int64_t table_stride(const Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }
void angle_table(const Tensor &t) {
  here(t, "table");
  if (t.dim() != 3 || t.size(2) != 2 || t.scalar_type() != at::kFloat || !t.is_contiguous())
    bad("table must be a contiguous fp32 CUDA tensor [positions, rot / 2, 2]");
}
// an output with the shape and type of q: the caller's, or a new contiguous one
Tensor like(const Tensor *out, const Tensor &q) {
  if (!out) return at::empty(q.sizes(), q.options());
  heads(*out, "out");
  written(*out, "out");
  same_type(*out, q, "out");
  if (out->sizes() != q.sizes()) bad("out must have the shape of q");
  return *out;
}
void *stream(const Tensor &t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }
Tensor bytes(size_t n, const Tensor &t) { return at::empty({(int64_t)n}, t.options().dtype(at::kByte)); }
// a workspace that the caller gives: its status word is read later, so it is used as it is or refused
void scratch(const Tensor &t, size_t need) {
  here(t, "workspace");
  if (!t.is_contiguous() || t.nbytes() < need) bad("workspace must be contiguous and have at least " + std::to_string(need) + " bytes");
}
// tells autograd that t has been written, so that a backward that saved what was there before fails instead of using this
void wrote(const Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void wrote(std::initializer_list<const Tensor *> ts) {
  for (const Tensor *t : ts)
    if (t) wrote(*t);
}
int32_t *i32(const Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); }
const int32_t *i32(const Tensor *t) { return t ? static_cast<const int32_t *>(t->data_ptr()) : nullptr; }
const void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

gdn_paged_shape paged_shape(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &table, const Tensor &lens, const Tensor *cu) {
  heads(q, "q");
  if (k.dim() != 4 || v.sizes() != k.sizes()) bad("k_cache and v_cache must have one shape [pages, page_size, kv heads, features]");
  features(k, "k_cache");
  features(v, "v_cache");
  gdn_paged_shape s = {};
  s.dtype = dtype(q, "q");
  same_type(k, q, "k_cache");
  same_type(v, q, "v_cache");
  if (k.size(3) != q.size(2)) bad("q and the caches must have the same number of features");
  page_table(table);
  const int64_t n = table.size(0);
  ints(lens, "kv_lens", n);
  if (cu) ints(*cu, "cu_q", n + 1);
  s.num_seqs = fits(n, "the number of sequences");
  s.total_q = fits(q.size(0), "the number of new tokens");
  s.num_heads = fits(q.size(1), "the number of heads");
  s.num_kv_heads = fits(k.size(2), "the number of kv heads");
  s.head_dim = fits(q.size(2), "the number of features");
  s.num_pages = fits(k.size(0), "the number of pages");
  s.page_size = fits(k.size(1), "the page size");
  s.max_pages = fits(table.size(1), "the width of page_table");
  s.table_stride = table_stride(table);
  s.q_tok = q.stride(0);
  s.q_head = q.stride(1);
  s.k_page = k.stride(0);
  s.k_tok = k.stride(1);
  s.k_head = k.stride(2);
  s.v_page = v.stride(0);
  s.v_tok = v.stride(1);
  s.v_head = v.stride(2);
  return s;
}

// ------------------------------------------------------------------ results
PyObject *pack(std::initializer_list<Tensor> ts) {
  PyObject *t = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const Tensor &x : ts) {
    if (x.defined()) {
      PyTuple_SET_ITEM(t, i++, THPVariable_Wrap(x));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(t, i++, Py_None);
    }
  }
  return t;
}

// ------------------------------------------------------------------ the functions
// q, k_cache, v_cache, page_table, kv_lens, cu_q, max_q, scale, window, return_lse, out, workspace
PyObject *paged_attention(PyObject *const *a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache"), &table = tensor(a[3], "page_table"),
               &lens = tensor(a[4], "kv_lens");
  const Tensor *cu = maybe(a[5], "cu_q"), *out = maybe(a[10], "out"), *given = maybe(a[11], "workspace");
  gdn_paged_shape s = paged_shape(q, k, v, table, lens, cu);
  s.max_q = small_int(a[6], "max_q");
  s.scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)q.size(2))) : (float)number(a[7]);
  s.window = small_int(a[8], "window");
  const Tensor o = like(out, q);
  s.o_tok = o.stride(0);
  s.o_head = o.stride(1);
  const size_t need = api.paged_attn_workspace_size(&s);
  if (!need) check(GDN_ERR_INVALID_ARG, "gdn_paged_attn_workspace_size");
  Tensor lse;
  if (truth(a[9])) lse = at::empty({q.size(0), q.size(1)}, q.options().dtype(at::kFloat));
  if (given) scratch(*given, need);
  const Tensor ws = given ? *given : bytes(need, q);
  check(api.paged_attn_fwd(&s, q.data_ptr(), k.data_ptr(), v.data_ptr(), i32(table), i32(cu), i32(lens), o.data_ptr(),
                           lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr, ws.data_ptr(), ws.nbytes(),
                           (gdn_stream_t)stream(q)),
        "gdn_paged_attn_fwd");
  wrote({out});
  return lse.defined() ? pack({o, lse}) : THPVariable_Wrap(o);
}

// q, k_cache, v_cache, page_table, kv_lens, workspace, cu_q, max_q
PyObject *paged_attention_status(PyObject *const *a) {
  const Tensor &q = tensor(a[0], "q"), &ws = tensor(a[5], "workspace");
  gdn_paged_shape s = paged_shape(q, tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), tensor(a[3], "page_table"), tensor(a[4], "kv_lens"),
                                  maybe(a[6], "cu_q"));
  s.max_q = small_int(a[7], "max_q");
  s.scale = 1.f;
  s.o_tok = q.size(1) * q.size(2);
  s.o_head = q.size(2);
  const size_t need = api.paged_attn_workspace_size(&s);
  if (!need) check(GDN_ERR_INVALID_ARG, "gdn_paged_attn_workspace_size");
  scratch(ws, need);
  return PyLong_FromLong(api.paged_attn_status(&s, ws.data_ptr(), (gdn_stream_t)stream(q)));
}

// q, k, table, positions, interleaved, inverse, inplace
PyObject *rotary(PyObject *const *a) {
  const Tensor &q = tensor(a[0], "q"), &table = tensor(a[2], "table"), &pos = tensor(a[3], "positions");
  const Tensor *k = maybe(a[1], "k");
  const bool inplace = truth(a[6]);
  heads(q, "q");
  angle_table(table);
  gdn_rotary_shape s = {};
  s.dtype = dtype(q, "q");
  ints(pos, "positions", q.size(0));
  s.tokens = fits(q.size(0), "the number of tokens");
  s.q_heads = fits(q.size(1), "the number of heads");
  s.head_dim = fits(q.size(2), "the number of features");
  s.rot = fits(2 * table.size(1), "rot");
  s.table_rows = fits(table.size(0), "the table");
  s.interleaved = truth(a[4]);
  s.inverse = truth(a[5]);
  if (inplace) written(q, "q");
  if (inplace && k) written(*k, "k");
  const Tensor qo = inplace ? q : at::empty(q.sizes(), q.options());
  s.q_tok = q.stride(0);
  s.q_head = q.stride(1);
  s.qo_tok = qo.stride(0);
  s.qo_head = qo.stride(1);
  Tensor ko;
  if (k) {
    heads(*k, "k");
    same_type(*k, q, "k");
    if (k->size(0) != q.size(0) || k->size(2) != q.size(2)) bad("q and k must have the same tokens and features");
    ko = inplace ? *k : at::empty(k->sizes(), k->options());
    s.k_heads = fits(k->size(1), "the number of heads");
    s.k_tok = k->stride(0);
    s.k_head = k->stride(1);
    s.ko_tok = ko.stride(0);
    s.ko_head = ko.stride(1);
  }
  check(api.rotary(&s, q.data_ptr(), ptr(k), static_cast<const float *>(table.data_ptr()), i32(pos), qo.data_ptr(),
                   ko.defined() ? ko.data_ptr() : nullptr, (gdn_stream_t)stream(q)),
        "gdn_rotary");
  if (inplace) wrote({&q, k});
  return pack({qo, ko});
}

// q, k, v, table, k_cache, v_cache, page_table, kv_lens, cu_q, interleaved, out
PyObject *rotary_append(PyObject *const *a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &table = tensor(a[3], "table"),
               &kc = tensor(a[4], "k_cache"), &vc = tensor(a[5], "v_cache"), &pages = tensor(a[6], "page_table"), &lens = tensor(a[7], "kv_lens");
  const Tensor *cu = maybe(a[8], "cu_q"), *out = maybe(a[10], "out");
  gdn_paged_shape s = paged_shape(q, kc, vc, pages, lens, cu);
  written(kc, "k_cache");
  written(vc, "v_cache");
  heads(k, "k");
  heads(v, "v");
  same_type(k, q, "k");
  same_type(v, q, "v");
  if (k.size(0) != q.size(0) || k.size(1) != kc.size(2) || k.size(2) != q.size(2) || v.sizes() != k.sizes())
    bad("k and v must be [new tokens, kv heads, features]");
  angle_table(table);
  const Tensor o = like(out, q);
  s.o_tok = o.stride(0);
  s.o_head = o.stride(1);
  s.kn_tok = k.stride(0);
  s.kn_head = k.stride(1);
  s.vn_tok = v.stride(0);
  s.vn_head = v.stride(1);
  s.rot = fits(2 * table.size(1), "rot");
  s.table_rows = fits(table.size(0), "the table");
  s.interleaved = truth(a[9]);
  check(api.rotary_append(&s, q.data_ptr(), k.data_ptr(), v.data_ptr(), static_cast<const float *>(table.data_ptr()), kc.data_ptr(),
                          vc.data_ptr(), i32(pages), i32(cu), i32(lens), o.data_ptr(), (gdn_stream_t)stream(q)),
        "gdn_rotary_append");
  wrote({&kc, &vc, out});
  return THPVariable_Wrap(o);
}

// the pools of a call, and the tensors that hold them
struct Pools {
  std::vector<gdn_slot_pool> p;
  std::vector<Tensor> held;
  const gdn_slot_pool *data() const { return p.data(); }
  int size() const { return (int)p.size(); }
  void wrote_all() const {
    for (const Tensor &t : held) wrote(t);
  }
};
// least: slots that each has to have
Pools pools(PyObject *seq, const char *name, int64_t least) {
  PyObject *fast = PySequence_Fast(seq, "pools must be a sequence of tensors");
  if (!fast) throw std::invalid_argument("");
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
  Pools r;
  try {
    for (Py_ssize_t i = 0; i < n; ++i) {
      const Tensor &t = tensor(PySequence_Fast_GET_ITEM(fast, i), name);
      if (t.dim() < 1) bad(std::string(name) + " must be tensors of slots");
      here(t, name);
      const int64_t slots = t.size(0);
      if (slots < least) bad(std::string(name) + " must have " + std::to_string(least) + " slots or more (the first dimension counts them)");
      int64_t inner = t.element_size(), want = 1;
      for (int64_t d = t.dim() - 1; d > 0; --d) {  // a slot's values lie in one piece
        if (slots && t.size(d) > 1 && t.stride(d) != want) bad(std::string("each slot of ") + name + " must be contiguous");
        want *= t.size(d);
      }
      inner *= slots ? want : 0;
      // an empty pool has no address: it has nothing to copy either
      if (inner > 0) r.p.push_back({t.data_ptr(), slots > 1 ? t.stride(0) * (int64_t)t.element_size() : inner, inner, slots});
      r.held.push_back(t);
    }
  } catch (...) {
    Py_DECREF(fast);
    throw;
  }
  Py_DECREF(fast);
  return r;
}

gdn_pages_shape pages_shape(const Tensor &table, const Tensor &ref, int page_size) {
  page_table(table);
  ints(ref, "refcount");
  gdn_pages_shape s = {};
  s.num_seqs = fits(table.size(0), "the number of sequences");
  s.max_pages = fits(table.size(1), "the width of page_table");
  s.num_pages = fits(ref.numel(), "the number of pages");
  s.page_size = page_size;
  s.table_stride = table_stride(table);
  return s;
}
Tensor pages_workspace(const gdn_pages_shape &s, int m, const Tensor &t) {
  const size_t need = api.pages_workspace_size(&s, m);
  if (!need) check(GDN_ERR_INVALID_ARG, "gdn_pages_workspace_size");
  return bytes(need, t);
}

// page_table, seq_lens, refcount, seqs, add, page_size
PyObject *extend_pages(PyObject *const *a) {
  const Tensor &table = tensor(a[0], "page_table"), &lens = tensor(a[1], "seq_lens"), &ref = tensor(a[2], "refcount"),
               &seqs = tensor(a[3], "seqs"), &add = tensor(a[4], "add");
  const gdn_pages_shape s = pages_shape(table, ref, small_int(a[5], "page_size"));
  ints(lens, "seq_lens", s.num_seqs);
  ints(seqs, "seqs");
  ints(add, "add", seqs.numel());
  const int m = fits(seqs.numel(), "the number of requests");
  const Tensor ok = at::empty_like(seqs), ws = pages_workspace(s, m, seqs);
  check(api.pages_extend(&s, i32(table), i32(lens), i32(ref), i32(seqs), i32(add), m, i32(ok), ws.data_ptr(), ws.nbytes(),
                         (gdn_stream_t)stream(seqs)),
        "gdn_pages_extend");
  wrote({&table, &lens, &ref});
  return THPVariable_Wrap(ok);
}

// page_table, seq_lens, refcount, parents, children, pools, page_size, states
PyObject *fork_pages(PyObject *const *a) {
  const Tensor &table = tensor(a[0], "page_table"), &lens = tensor(a[1], "seq_lens"), &ref = tensor(a[2], "refcount"),
               &par = tensor(a[3], "parents"), &chi = tensor(a[4], "children");
  const gdn_pages_shape s = pages_shape(table, ref, small_int(a[6], "page_size"));
  ints(lens, "seq_lens", s.num_seqs);
  ints(par, "parents");
  ints(chi, "children", par.numel());
  const Pools p = pools(a[5], "pools", s.num_pages), st = pools(a[7], "states", s.num_seqs);
  const int m = fits(par.numel(), "the number of forks");
  const Tensor fresh = at::empty_like(par), ws = pages_workspace(s, m, par);
  check(api.pages_fork(&s, i32(table), i32(lens), i32(ref), i32(par), i32(chi), m, p.data(), p.size(), st.data(), st.size(),
                       i32(fresh), ws.data_ptr(), ws.nbytes(), (gdn_stream_t)stream(par)),
        "gdn_pages_fork");
  wrote({&table, &lens, &ref});
  p.wrote_all();
  st.wrote_all();
  return THPVariable_Wrap(fresh);
}

// page_table, seq_lens, refcount, seqs
PyObject *free_pages(PyObject *const *a) {
  const Tensor &table = tensor(a[0], "page_table"), &lens = tensor(a[1], "seq_lens"), &ref = tensor(a[2], "refcount"), &seqs = tensor(a[3], "seqs");
  const gdn_pages_shape s = pages_shape(table, ref, 1);
  ints(lens, "seq_lens", s.num_seqs);
  ints(seqs, "seqs");
  check(api.pages_free(&s, i32(table), i32(lens), i32(ref), i32(seqs), fits(seqs.numel(), "the number of sequences"),
                       (gdn_stream_t)stream(seqs)),
        "gdn_pages_free");
  wrote({&table, &lens, &ref});
  Py_RETURN_NONE;
}

// page_table, refcount, pools, inplace
PyObject *compact_pages(PyObject *const *a) {
  const Tensor &table = tensor(a[0], "page_table"), &ref = tensor(a[1], "refcount");
  const gdn_pages_shape s = pages_shape(table, ref, 1);
  const Pools p = pools(a[2], "pools", s.num_pages);
  const bool inplace = truth(a[3]);
  const Tensor t = inplace ? table : at::empty_strided(table.sizes(), {s.table_stride, 1}, table.options());
  const Tensor r = inplace ? ref : at::empty_like(ref);
  const Tensor moves = at::empty({}, ref.options()), ws = pages_workspace(s, 0, ref);
  check(api.pages_compact(&s, i32(table), i32(ref), i32(t), i32(r), p.data(), p.size(), i32(moves), ws.data_ptr(), ws.nbytes(),
                          (gdn_stream_t)stream(ref)),
        "gdn_pages_compact");
  if (inplace) wrote({&table, &ref});
  p.wrote_all();
  return pack({t, r, moves});
}

// pools, src, dst
PyObject *copy_slots(PyObject *const *a) {
  const Tensor &src = tensor(a[1], "src"), &dst = tensor(a[2], "dst");
  ints(src, "src");
  ints(dst, "dst", src.numel());
  const Pools p = pools(a[0], "pools", 0);
  check(api.slots_copy(p.data(), p.size(), i32(src), i32(dst), fits(src.numel(), "the number of pairs"), (gdn_stream_t)stream(src)),
        "gdn_slots_copy");
  p.wrote_all();
  Py_RETURN_NONE;
}

// the common stride of the rows of t [..., dim], as if it had two dimensions
int64_t row_stride(const Tensor &t, const char *name) {
  const int64_t dim = t.size(-1);
  if (t.dim() == 1) return dim;
  int64_t stride = 0, want = 0;
  bool set = false;
  for (int64_t d = t.dim() - 2; d >= 0; --d) {
    if (t.size(d) == 1) continue;
    if (!set) {
      stride = t.stride(d);
      set = true;
    } else if (t.stride(d) != want) {
      bad(std::string("the rows of ") + name + " must have one stride");
    }
    want = t.stride(d) * t.size(d);
  }
  return set ? stride : dim;
}
const Tensor &norm_weight(const Tensor &w, int64_t dim) {
  if (w.scalar_type() != at::kFloat || w.dim() != 1 || w.size(0) != dim || !w.is_contiguous())
    bad("weight must be a contiguous fp32 CUDA tensor [dim]");
  here(w, "weight");
  return w;
}
void same_as(const Tensor &t, const Tensor &x, const char *name) {
  features(t, name);
  same_type(t, x, name);
  if (t.sizes() != x.sizes()) bad(std::string(name) + " must have the shape of the other inputs");
}

// x, weight, residual, eps, fp8, group, weight_offset, inplace -> (y, h, scale, rstd)
PyObject *rms_norm(PyObject *const *a) {
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
  const Tensor *res = maybe(a[2], "residual");
  const bool fp8 = truth(a[4]), inplace = truth(a[7]);
  features(x, "x");
  const int64_t dim = x.size(-1), rows = dim ? x.numel() / dim : 0;
  gdn_norm_shape s = {};
  s.rows = rows;
  s.dim = fits(dim, "dim");
  s.dtype = dtype(x, "x");
  s.fp8 = fp8;
  s.group = small_int(a[5], "group");
  s.eps = (float)number(a[3]);
  s.weight_offset = (float)number(a[6]);
  s.x_row = row_stride(x, "x");
  s.y_row = dim;
  norm_weight(w, dim);
  Tensor h = x;
  if (res) {
    same_as(*res, x, "residual");
    s.r_row = row_stride(*res, "residual");
    h = inplace ? *res : at::empty(x.sizes(), x.options());
    s.h_row = inplace ? s.r_row : dim;
  }
  const Tensor y = at::empty(x.sizes(), fp8 ? x.options().dtype(at::kFloat8_e4m3fn) : x.options());
  const c10::IntArrayRef lead = x.sizes().slice(0, (size_t)x.dim() - 1);
  const Tensor rstd = at::empty(lead, x.options().dtype(at::kFloat));
  Tensor scale;
  if (fp8) {
    c10::SmallVector<int64_t, 6> size(lead.begin(), lead.end());
    size.push_back(s.group > 0 ? dim / s.group : 1);
    scale = at::empty(size, rstd.options());
  }
  check(api.rmsnorm_fwd(&s, x.data_ptr(), ptr(res), static_cast<const float *>(w.data_ptr()), res ? h.data_ptr() : nullptr, y.data_ptr(),
                        fp8 ? static_cast<float *>(scale.data_ptr()) : nullptr, static_cast<float *>(rstd.data_ptr()),
                        (gdn_stream_t)stream(x)),
        "gdn_rmsnorm_fwd");
  if (inplace) wrote({res});
  return pack({y, h, scale, rstd});
}

// dy, h, weight, rstd, dh, weight_offset -> (dx, dw)
PyObject *rms_norm_bwd(PyObject *const *a) {
  const Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h"), &w = tensor(a[2], "weight"), &rstd = tensor(a[3], "rstd");
  const Tensor *dh = maybe(a[4], "dh");
  features(dy, "dy");
  same_as(h, dy, "h");
  const int64_t dim = dy.size(-1), rows = dim ? dy.numel() / dim : 0;
  gdn_norm_shape s = {};
  s.rows = rows;
  s.dim = fits(dim, "dim");
  s.dtype = dtype(dy, "dy");
  s.weight_offset = (float)number(a[5]);
  s.x_row = row_stride(h, "h");
  s.y_row = row_stride(dy, "dy");
  s.h_row = dim;
  norm_weight(w, dim);
  here(rstd, "rstd");
  if (rstd.scalar_type() != at::kFloat || rstd.numel() != rows || !rstd.is_contiguous())
    bad("rstd must be a contiguous fp32 tensor with one value per row");
  if (dh) {
    same_as(*dh, dy, "dh");
    s.r_row = row_stride(*dh, "dh");
  }
  const Tensor dx = at::empty(dy.sizes(), dy.options()), dw = at::empty({dim}, w.options());
  const size_t need = api.rmsnorm_bwd_workspace_size(&s);
  if (!need) check(GDN_ERR_INVALID_ARG, "gdn_rmsnorm_bwd_workspace_size");
  const Tensor ws = bytes(need, dy);
  check(api.rmsnorm_bwd(&s, dy.data_ptr(), h.data_ptr(), static_cast<const float *>(w.data_ptr()),
                        static_cast<const float *>(rstd.data_ptr()), ptr(dh), dx.data_ptr(), static_cast<float *>(dw.data_ptr()),
                        ws.data_ptr(), ws.nbytes(), (gdn_stream_t)stream(dy)),
        "gdn_rmsnorm_bwd");
  return pack({dx, dw});
}

// addresses of the C entry points, in the order of Api
PyObject *connect(PyObject *const *a) {
  void **slot = reinterpret_cast<void **>(&api);
  for (size_t i = 0; i < sizeof(Api) / sizeof(void *); ++i) {
    slot[i] = PyLong_AsVoidPtr(a[i]);
    if (!slot[i]) bad("connect needs the address of every entry point");
  }
  connected = true;
  Py_RETURN_NONE;
}

// Positional arguments only; nothing thrown here leaves as a C++ exception.
template <PyObject *(*F)(PyObject *const *), int N> PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    if (!connected && F != connect) throw std::runtime_error("the CUDA library is not connected");
    return F(args);
  } catch (const ValueError &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError &e) {  // of an output or a workspace: callers may free memory and try again
    PyObject *torch = PyImport_ImportModule("torch"), *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}
#define ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}

PyMethodDef methods[] = {ENTRY(connect, (int)(sizeof(Api) / sizeof(void *))),
                         ENTRY(paged_attention, 12),
                         ENTRY(paged_attention_status, 8),
                         ENTRY(rotary, 7),
                         ENTRY(rotary_append, 11),
                         ENTRY(extend_pages, 6),
                         ENTRY(fork_pages, 8),
                         ENTRY(free_pages, 4),
                         ENTRY(compact_pages, 4),
                         ENTRY(copy_slots, 3),
                         ENTRY(rms_norm, 8),
                         ENTRY(rms_norm_bwd, 6),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdn_block_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gdn_block_py(void) { return PyModule_Create(&module); }
