// paged_binding.cpp -- Python side of the paged-cache and output-layer calls (module _paged_calls): checks the
// tensors, allocates the results and calls the C ABI of libfatattn.so. A decode step is bound by the
// host's time per call, and the same checks in Python cost 10 to 20 us a call on the host cores (25 us
// against 10 for a one-token attention step). The public functions, with their documentation, are
// those of the package; they pass their arguments on in order and raise the library's errors.
// Nothing here computes: every value comes from the library's kernels.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>

#include <optional>

#include "../../include/fat_attn.h"

namespace {

decltype(&fat_paged_plan) p_plan;
decltype(&fat_rope_embed) p_rope;
decltype(&fat_paged_append) p_append;
decltype(&fat_paged_attn) p_attn;
decltype(&fat_paged_attn_workspace_size) p_attn_ws;
decltype(&fat_paged_tree_plan) p_tree_plan;
decltype(&fat_paged_tree_attn) p_tree_attn;
decltype(&fat_linear_cross_entropy_fwd) p_lce_fwd;
decltype(&fat_linear_cross_entropy_bwd) p_lce_bwd;
decltype(&fat_linear_cross_entropy_workspace_size) p_lce_ws;
PyObject *g_rope_type;  // the Python class of fat_rope_t records

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(PyObject *type, const char *fmt, const char *name, const char *what = "") {
  PyErr_Format(type, fmt, name, what);
  throw Refused{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// A tensor argument's type and device (dev < 0: it gives the device).
void check(const at::Tensor &t, const char *name, at::ScalarType type, int dev) {
  if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s", name, c10::toString(type));
  if (!t.is_cuda() || (dev >= 0 && t.get_device() != dev))
    refuse(PyExc_ValueError, "%s must be a CUDA tensor on the device of the other arguments", name);
}
void check_rank(const at::Tensor &t, const char *name, int64_t rank) {
  if (t.dim() != rank) refuse(PyExc_ValueError, "%s must have another number of dimensions", name);
}
void check_shape(const at::Tensor &t, const char *name, at::IntArrayRef shape) {
  if (t.sizes() != shape) refuse(PyExc_ValueError, "%s does not have the shape of the call", name);
}
void check_contiguous(const at::Tensor &t, const char *name) {
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
}
// bf16 rows with a contiguous last dimension
void check_rows(const at::Tensor &t, const char *name, int64_t rank, int dev) {
  check(t, name, at::kBFloat16, dev);
  check_rank(t, name, rank);
  if (t.stride(rank - 1) != 1 && t.size(rank - 1) > 1)
    refuse(PyExc_ValueError, "%s: the last dimension must be contiguous", name);
}
int32_t *ints(PyObject *o, const char *name, int64_t numel, int dev) {
  const at::Tensor &t = tensor(o, name);
  check(t, name, at::kInt, dev);
  check_contiguous(t, name);
  if (numel >= 0 && t.numel() != numel)
    refuse(PyExc_ValueError, "%s does not have the number of entries of the call", name);
  return static_cast<int32_t *>(t.data_ptr());
}
const float *floats(PyObject *o, const char *name, at::IntArrayRef shape, int dev) {
  const at::Tensor &t = tensor(o, name);
  check(t, name, at::kFloat, dev);
  check_shape(t, name, shape);
  check_contiguous(t, name);
  return static_cast<const float *>(t.data_ptr());
}
int32_t integer(PyObject *o, const char *name) {
  PyObject *i = PyNumber_Index(o);
  if (!i) throw Refused{};
  const long long v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s is out of range", name);
  return (int32_t)v;
}
int32_t small(int64_t v, const char *name) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, "%s is too large", name);
  return (int32_t)v;
}
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}
// The call's stream. A given one is the current one while this lives: results and workspaces are
// allocated on it, so that their memory is taken and given back in its order.
struct OnStream {
  c10::cuda::OptionalCUDAStreamGuard guard;
  void *stream;
  OnStream(PyObject *o, int dev) {
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      return;
    }
    stream = PyLong_AsVoidPtr(o);
    if (!stream && PyErr_Occurred()) throw Refused{};
    guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream),
                                                        (c10::DeviceIndex)dev));
  }
};
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
}
fat_paged_cache_t cache_of(PyObject *ko, PyObject *vo, int dev) {
  const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
  check_rows(k, "k_cache", 4, dev);
  check_rows(v, "v_cache", 4, dev);
  check_shape(v, "v_cache", k.sizes());
  for (int64_t i = 0; i < 3; ++i)  // a stride over one entry says nothing
    if (v.stride(i) != k.stride(i) && k.size(i) > 1)
      refuse(PyExc_ValueError, "%s must have the strides of k_cache", "v_cache");
  fat_paged_cache_t c;
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.num_pages = small(k.size(0), "k_cache");
  c.page_size = small(k.size(1), "k_cache");
  c.num_heads = small(k.size(2), "k_cache");
  c.head_dim = small(k.size(3), "k_cache");
  c.stride_page = k.stride(0);
  c.stride_token = k.stride(1);
  c.stride_head = k.stride(2);
  return c;
}

// A fat_rope_t record of the package's class, or null for None.
struct Rope {
  Py_buffer view{};
  explicit Rope(PyObject *o) {
    if (o == Py_None) return;
    if ((PyObject *)Py_TYPE(o) != g_rope_type)
      refuse(PyExc_TypeError, "%s must come from fat_rope_init", "rope");
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE)) throw Refused{};
    if (view.len != (Py_ssize_t)sizeof(fat_rope_t)) {
      PyBuffer_Release(&view);
      refuse(PyExc_TypeError, "%s must come from fat_rope_init", "rope");
    }
  }
  ~Rope() {
    if (view.obj) PyBuffer_Release(&view);
  }
  Rope(const Rope &) = delete;
  const fat_rope_t *get() const { return static_cast<const fat_rope_t *>(view.buf); }
};

// Run a library call on device dev without the interpreter's lock.
template <typename F>
int call_on(int dev, F f) {
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

#define ENTRY(name, count)                                                            \
  PyObject *name(PyObject *, PyObject *const *a, Py_ssize_t n) {                      \
    HANDLE_TH_ERRORS                                                                  \
    if (n != count) return PyErr_Format(PyExc_TypeError, "%d arguments", (int)count); \
    try {
#define ENTRY_END             \
  }                           \
  catch (const Refused &) {   \
    return nullptr;           \
  }                           \
  END_HANDLE_TH_ERRORS        \
  }

// Results: a tuple, or the library's error code.

// ctx_lens, new_lens, free_pages, block_table, page_size, num_pages, max_tokens, cu_seqlens_q,
// seqlens_k, positions, slots, counts, stream
ENTRY(plan, 13)
  const at::Tensor &ctx = tensor(a[0], "ctx_lens"), &table = tensor(a[3], "block_table");
  check(ctx, "ctx_lens", at::kInt, -1);
  const int dev = ctx.get_device();
  const int64_t num = ctx.numel();
  check_rank(table, "block_table", 2);
  if (table.size(0) != num)
    refuse(PyExc_ValueError, "%s must have a row for every request", "block_table");
  const int32_t max_tokens = integer(a[6], "max_tokens");
  fat_plan_shape_t sh{};
  sh.num_seqs = small(num, "ctx_lens");
  sh.page_size = integer(a[4], "page_size");
  sh.num_pages = integer(a[5], "num_pages");
  sh.table_width = small(table.size(1), "block_table");
  const int32_t *pc = ints(a[0], "ctx_lens", num, dev), *pn = ints(a[1], "new_lens", num, dev);
  const int32_t *pf = ints(a[2], "free_pages", -1, dev);
  sh.num_free = small(tensor(a[2], "free_pages").numel(), "free_pages");
  sh.max_tokens = max_tokens;
  int32_t *pt = ints(a[3], "block_table", -1, dev);
  const OnStream on(a[12], dev);
  sh.stream = on.stream;
  static const char *const names[5] = {"cu_seqlens_q", "seqlens_k", "positions", "slots", "counts"};
  const int64_t sizes[5] = {num + 1, num, max_tokens < 0 ? 0 : max_tokens,
                            max_tokens < 0 ? 0 : max_tokens, 2};
  at::Tensor made[5];
  int32_t *out[5];
  for (int i = 0; i < 5; ++i) {
    if (a[7 + i] == Py_None) {
      made[i] = make({sizes[i]}, at::kInt, dev);
      out[i] = static_cast<int32_t *>(made[i].data_ptr());
    } else {
      out[i] = ints(a[7 + i], names[i], sizes[i], dev);
    }
  }
  const int rc = call_on(
      dev, [&] { return p_plan(&sh, pc, pn, pf, pt, out[0], out[1], out[2], out[3], out[4]); });
  if (rc) return PyLong_FromLong(rc);
  PyObject *res = PyTuple_New(5);
  if (!res) return nullptr;
  for (int i = 0; i < 5; ++i) {
    PyObject *o = made[i].defined() ? THPVariable_Wrap(made[i]) : Py_NewRef(a[7 + i]);
    PyTuple_SET_ITEM(res, i, o);
  }
  return res;
ENTRY_END

// x, positions, rope, inverse, out, stream
ENTRY(rope, 6)
  const at::Tensor &x = tensor(a[0], "x");
  check_rows(x, "x", 3, -1);
  const int dev = x.get_device();
  const Rope rope(a[2]);
  const OnStream on(a[5], dev);
  at::Tensor made;
  if (a[4] == Py_None) made = make(x.sizes(), at::kBFloat16, dev);
  const at::Tensor &y = made.defined() ? made : tensor(a[4], "out");
  check_rows(y, "out", 3, dev);
  check_shape(y, "out", x.sizes());
  fat_rope_shape_t sh{};
  sh.tokens = small(x.size(0), "x");
  sh.num_heads = small(x.size(1), "x");
  sh.head_dim = small(x.size(2), "x");
  sh.x_stride_token = x.stride(0);
  sh.x_stride_head = x.stride(1);
  sh.y_stride_token = y.stride(0);
  sh.y_stride_head = y.stride(1);
  sh.stream = on.stream;
  const int32_t *pos = ints(a[1], "positions", x.size(0), dev);
  const int inverse = truth(a[3]) ? 1 : 0;
  const int rc = call_on(
      dev, [&] { return p_rope(&sh, rope.get(), x.data_ptr(), y.data_ptr(), pos, inverse); });
  if (rc) return PyLong_FromLong(rc);
  return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[4]);
ENTRY_END

// k, v, k_cache, v_cache, slots, q, positions, rope, q_out, stream
ENTRY(append, 10)
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  check_rows(k, "k", 3, -1);
  const int dev = k.get_device();
  const fat_paged_cache_t c = cache_of(a[2], a[3], dev);
  const int64_t T = k.size(0), d = c.head_dim;
  check_shape(k, "k", {T, c.num_heads, d});
  check_rows(v, "v", 3, dev);
  check_shape(v, "v", k.sizes());
  const Rope rope(a[7]);
  fat_append_shape_t sh{};
  sh.tokens = small(T, "k");
  sh.k_stride_token = k.stride(0);
  sh.k_stride_head = k.stride(1);
  sh.v_stride_token = v.stride(0);
  sh.v_stride_head = v.stride(1);
  const OnStream on(a[9], dev);
  sh.stream = on.stream;
  const void *pq = nullptr;
  void *po = nullptr;
  at::Tensor made;
  if (a[5] != Py_None) {
    const at::Tensor &q = tensor(a[5], "q");
    check_rows(q, "q", 3, dev);
    check_shape(q, "q", {T, q.size(1), d});
    sh.num_heads_q = small(q.size(1), "q");
    sh.q_stride_token = q.stride(0);
    sh.q_stride_head = q.stride(1);
    if (a[8] == Py_None) made = make(q.sizes(), at::kBFloat16, dev);
    const at::Tensor &y = made.defined() ? made : tensor(a[8], "q_out");
    check(y, "q_out", at::kBFloat16, dev);
    check_shape(y, "q_out", q.sizes());
    check_contiguous(y, "q_out");
    pq = q.data_ptr();
    po = y.data_ptr();
  } else if (a[8] != Py_None) {
    refuse(PyExc_ValueError, "%s is given without q", "q_out");
  }
  const int32_t *slots = ints(a[4], "slots", T, dev);
  const int32_t *pos = a[6] == Py_None ? nullptr : ints(a[6], "positions", T, dev);
  const int rc = call_on(dev, [&] {
    return p_append(&sh, &c, rope.get(), pq, k.data_ptr(), v.data_ptr(), pos, slots, po);
  });
  if (rc) return PyLong_FromLong(rc);
  PyObject *res = PyTuple_New(1);
  if (!res) return nullptr;
  PyTuple_SET_ITEM(res, 0, made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[8]));
  return res;
ENTRY_END

fat_paged_shape_t attn_shape(const at::Tensor &q, int64_t seqs, int64_t width, PyObject *max_q,
                             PyObject *max_k, void *stream) {
  fat_paged_shape_t sh{};
  sh.total_q = small(q.size(0), "q");
  sh.num_seqs = small(seqs, "seqlens_k");
  sh.max_seqlen_q = integer(max_q, "max_seqlen_q");
  sh.max_seqlen_k = integer(max_k, "max_seqlen_k");
  sh.num_heads_q = small(q.size(1), "q");
  sh.table_width = small(width, "block_table");
  sh.stream = stream;
  return sh;
}

// q, k_cache, cu_seqlens_q, max_seqlen_q, max_seqlen_k
ENTRY(attn_workspace, 5)
  const at::Tensor &q = tensor(a[0], "q");
  check_rows(q, "q", 3, -1);
  const int dev = q.get_device();
  const fat_paged_cache_t c = cache_of(a[1], a[1], dev);
  const fat_paged_shape_t sh =
      attn_shape(q, tensor(a[2], "cu_seqlens_q").numel() - 1, 0, a[3], a[4], nullptr);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  return PyLong_FromSize_t(p_attn_ws(&sh, &c));
ENTRY_END

// A given workspace, or one of the size that the call needs, made here.
struct Workspace {
  at::Tensor made;
  void *ptr;
  size_t bytes;
  template <typename F>
  Workspace(PyObject *o, int dev, F size) {
    if (o == Py_None) {
      const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
      bytes = size();
      made = make({(int64_t)bytes}, at::kByte, dev);
      ptr = made.data_ptr();
      return;
    }
    const at::Tensor &t = tensor(o, "workspace");
    if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
      refuse(PyExc_ValueError, "%s must be a contiguous CUDA tensor on the device of the call",
             "workspace");
    ptr = t.data_ptr();
    bytes = t.nbytes();
  }
};
// A result: the given tensor, or one made here.
struct Result {
  at::Tensor made;
  PyObject *given;
  void *ptr;
  Result(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType type, int dev) : given(o) {
    if (o == Py_None) {
      made = make(shape, type, dev);
      ptr = made.data_ptr();
      return;
    }
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, dev);
    check_shape(t, name, shape);
    check_contiguous(t, name);
    ptr = t.data_ptr();
  }
  PyObject *object() const { return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(given); }
};
PyObject *two(PyObject *a, PyObject *b) {
  PyObject *res = PyTuple_New(2);
  if (!res) return nullptr;
  PyTuple_SET_ITEM(res, 0, a);
  PyTuple_SET_ITEM(res, 1, b);
  return res;
}

// Both attention calls. a: q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k; b: max_seqlen_q,
// max_seqlen_k, bias_table, num_buckets, max_distance, bidirectional, alibi_slopes, then for
// fat_paged_attn causal, for both softmax_scale, out, lse, workspace, stream. tree: positions, tree_mask.
PyObject *attention(PyObject *const *a, PyObject *const *b, PyObject *const *tree) {
  const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "block_table");
  check_rows(q, "q", 3, -1);
  check_contiguous(q, "q");
  const int dev = q.get_device();
  const fat_paged_cache_t c = cache_of(a[1], a[2], dev);
  const int64_t Tq = q.size(0), Hq = q.size(1);
  if (q.size(2) != c.head_dim)
    refuse(PyExc_ValueError, "%s and the cache have different head dimensions", "q");
  check_rank(table, "block_table", 2);
  const int64_t num = tensor(a[5], "seqlens_k").numel();
  if (table.size(0) != num)
    refuse(PyExc_ValueError, "%s must have a row for every request", "block_table");
  const int32_t *pt = ints(a[3], "block_table", -1, dev);
  const int32_t *pcu = ints(a[4], "cu_seqlens_q", num + 1, dev);
  const int32_t *plk = ints(a[5], "seqlens_k", num, dev);
  const int32_t *pos = nullptr, *mask = nullptr;
  int32_t words = 0;
  if (tree) {
    pos = ints(tree[0], "positions", Tq, dev);
    const at::Tensor &t = tensor(tree[1], "tree_mask");
    check_rank(t, "tree_mask", 2);
    if (t.size(0) != Tq) refuse(PyExc_ValueError, "%s must have a row for every query", "tree_mask");
    mask = ints(tree[1], "tree_mask", -1, dev);
    words = small(t.size(1), "tree_mask");
  }
  const int32_t nb = integer(b[3], "num_buckets"), md = integer(b[4], "max_distance");
  const float *bias = b[2] == Py_None ? nullptr : floats(b[2], "bias_table", {nb, Hq}, dev);
  const float *slopes = b[6] == Py_None ? nullptr : floats(b[6], "alibi_slopes", {Hq}, dev);
  const int bidir = truth(b[5]) ? 1 : 0, causal = tree ? 0 : truth(b[7]) ? 1 : 0;
  PyObject *const *r = b + (tree ? 7 : 8);
  const float scale = (float)number(r[0]);
  const OnStream on(r[4], dev);
  const fat_paged_shape_t sh = attn_shape(q, num, table.size(1), b[0], b[1], on.stream);
  const Result out(r[1], "out", q.sizes(), at::kBFloat16, dev);
  const Result lse(r[2], "lse", {Hq, Tq}, at::kFloat, dev);
  const Workspace ws(r[3], dev, [&] { return p_attn_ws(&sh, &c); });
  const int rc = call_on(dev, [&] {
    if (tree)
      return p_tree_attn(&sh, &c, q.data_ptr(), pt, pcu, plk, pos, mask, words, bias, nb, md, bidir,
                         slopes, scale, ws.ptr, ws.bytes, out.ptr, static_cast<float *>(lse.ptr));
    return p_attn(&sh, &c, q.data_ptr(), pt, pcu, plk, bias, nb, md, bidir, slopes, causal, scale,
                  ws.ptr, ws.bytes, out.ptr, static_cast<float *>(lse.ptr));
  });
  if (rc) return PyLong_FromLong(rc);
  return two(out.object(), lse.object());
}

ENTRY(attn, 19)
  return attention(a, a + 6, nullptr);
ENTRY_END

// q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, positions, tree_mask, max_seqlen_q, ...
ENTRY(tree_attn, 20)
  return attention(a, a + 8, a + 6);
ENTRY_END

// parents, cu_seqlens_q, seqlens_k, max_seqlen_q, positions, tree_mask, stream
ENTRY(tree_plan, 7)
  const at::Tensor &par = tensor(a[0], "parents");
  check(par, "parents", at::kInt, -1);
  const int dev = par.get_device();
  const int64_t T = par.numel(), num = tensor(a[2], "seqlens_k").numel();
  const int32_t *pp = ints(a[0], "parents", -1, dev);
  const int32_t *pcu = ints(a[1], "cu_seqlens_q", num + 1, dev);
  const int32_t *plk = ints(a[2], "seqlens_k", num, dev);
  const int32_t most = integer(a[3], "max_seqlen_q");
  int64_t words = most < 0 ? 0 : (most + 31ll) / 32;
  if (a[5] != Py_None) {
    const at::Tensor &t = tensor(a[5], "tree_mask");
    check_rank(t, "tree_mask", 2);
    words = t.size(1);
  }
  const OnStream on(a[6], dev);
  const Result pos(a[4], "positions", {T}, at::kInt, dev);
  const Result mask(a[5], "tree_mask", {T, words}, at::kInt, dev);
  fat_tree_shape_t sh{};
  sh.total_q = small(T, "parents");
  sh.num_seqs = small(num, "seqlens_k");
  sh.max_seqlen_q = most;
  sh.mask_words = small(words, "tree_mask");
  sh.stream = on.stream;
  const int rc = call_on(dev, [&] {
    return p_tree_plan(&sh, pp, pcu, plk, static_cast<int32_t *>(pos.ptr),
                       static_cast<int32_t *>(mask.ptr));
  });
  if (rc) return PyLong_FromLong(rc);
  return two(pos.object(), mask.object());
ENTRY_END

// ---- output layer and loss
fat_linear_ce_shape_t head_shape(const at::Tensor &h, const at::Tensor &w, PyObject *z_loss,
                                 PyObject *logit_scale) {
  check_rows(h, "hidden", 2, -1);
  check_rows(w, "weight", 2, h.get_device());
  if (w.size(1) != h.size(1))
    refuse(PyExc_ValueError, "%s and hidden have different row lengths", "weight");
  fat_linear_ce_shape_t sh{};
  sh.rows = small(h.size(0), "hidden");
  sh.vocab = small(w.size(0), "weight");
  sh.dim = small(h.size(1), "hidden");
  // a stride over one row says nothing
  sh.hidden_stride = h.size(0) > 1 ? h.stride(0) : h.size(1);
  sh.weight_stride = w.size(0) > 1 ? w.stride(0) : w.size(1);
  sh.z_loss = (float)number(z_loss);
  sh.logit_scale = (float)number(logit_scale);
  return sh;
}
// rows, vocab, dim, backward
ENTRY(lce_workspace, 4)
  fat_linear_ce_shape_t sh{};
  sh.rows = integer(a[0], "rows");
  sh.vocab = integer(a[1], "vocab");
  sh.dim = integer(a[2], "dim");
  sh.hidden_stride = sh.weight_stride = sh.dim;
  sh.logit_scale = 1.f;
  return PyLong_FromSize_t(p_lce_ws(&sh, truth(a[3]) ? 1 : 0));
ENTRY_END

// hidden, weight, target, z_loss, logit_scale, loss, lse, workspace, stream
ENTRY(lce_fwd, 9)
  const at::Tensor &h = tensor(a[0], "hidden"), &w = tensor(a[1], "weight");
  fat_linear_ce_shape_t sh = head_shape(h, w, a[3], a[4]);
  const int dev = h.get_device();
  const int32_t *target = ints(a[2], "target", sh.rows, dev);
  const OnStream on(a[8], dev);
  sh.stream = on.stream;
  const Result loss(a[5], "loss", {sh.rows}, at::kFloat, dev);
  const Result lse(a[6], "lse", {sh.rows}, at::kFloat, dev);
  const Workspace ws(a[7], dev, [&] { return p_lce_ws(&sh, 0); });
  const int rc = call_on(dev, [&] {
    return p_lce_fwd(&sh, h.data_ptr(), w.data_ptr(), target, ws.ptr, ws.bytes,
                     static_cast<float *>(loss.ptr), static_cast<float *>(lse.ptr));
  });
  if (rc) return PyLong_FromLong(rc);
  return two(loss.object(), lse.object());
ENTRY_END

// hidden, weight, target, lse, dloss, z_loss, logit_scale, grad_scale, want_dhidden, want_dweight, dhidden,
// dweight, workspace, stream
ENTRY(lce_bwd, 14)
  const at::Tensor &h = tensor(a[0], "hidden"), &w = tensor(a[1], "weight");
  fat_linear_ce_shape_t sh = head_shape(h, w, a[5], a[6]);
  const int dev = h.get_device();
  const int32_t *target = ints(a[2], "target", sh.rows, dev);
  const float *lse = floats(a[3], "lse", {sh.rows}, dev);
  const float *dloss = a[4] == Py_None ? nullptr : floats(a[4], "dloss", {sh.rows}, dev);
  const float grad_scale = (float)number(a[7]);
  const bool want_h = truth(a[8]), want_w = truth(a[9]);
  if ((!want_h && a[10] != Py_None) || (!want_w && a[11] != Py_None))
    refuse(PyExc_ValueError, "%s is given but not wanted", want_h ? "dweight" : "dhidden");
  const OnStream on(a[13], dev);
  sh.stream = on.stream;
  std::optional<Result> dh, dw;
  if (want_h) dh.emplace(a[10], "dhidden", h.sizes(), at::kBFloat16, dev);
  if (want_w) dw.emplace(a[11], "dweight", w.sizes(), at::kBFloat16, dev);
  const Workspace ws(a[12], dev, [&] { return p_lce_ws(&sh, 1); });
  const int rc = call_on(dev, [&] {
    return p_lce_bwd(&sh, h.data_ptr(), w.data_ptr(), target, lse, dloss, grad_scale, ws.ptr, ws.bytes,
                     dh ? dh->ptr : nullptr, dw ? dw->ptr : nullptr);
  });
  if (rc) return PyLong_FromLong(rc);
  return two(dh ? dh->object() : Py_NewRef(Py_None), dw ? dw->object() : Py_NewRef(Py_None));
ENTRY_END

// path of libfatattn.so, class of the rotary records
ENTRY(bind, 2)
  const char *path = PyUnicode_AsUTF8(a[0]);
  if (!path) return nullptr;
  void *lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!lib) return PyErr_Format(PyExc_ImportError, "%s", dlerror());
#define BIND(p, name)                                                              \
  p = reinterpret_cast<decltype(p)>(dlsym(lib, name));                             \
  if (!p) return PyErr_Format(PyExc_ImportError, "%s has no %s", path, name)
  BIND(p_plan, "fat_paged_plan");
  BIND(p_rope, "fat_rope_embed");
  BIND(p_append, "fat_paged_append");
  BIND(p_attn, "fat_paged_attn");
  BIND(p_attn_ws, "fat_paged_attn_workspace_size");
  BIND(p_tree_plan, "fat_paged_tree_plan");
  BIND(p_tree_attn, "fat_paged_tree_attn");
  BIND(p_lce_fwd, "fat_linear_cross_entropy_fwd");
  BIND(p_lce_bwd, "fat_linear_cross_entropy_bwd");
  BIND(p_lce_ws, "fat_linear_cross_entropy_workspace_size");
#undef BIND
  Py_XSETREF(g_rope_type, Py_NewRef(a[1]));
  Py_RETURN_NONE;
ENTRY_END

#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(plan),           METHOD(rope), METHOD(append),
                         METHOD(attn_workspace), METHOD(attn), METHOD(lce_workspace),
                         METHOD(lce_fwd),        METHOD(lce_bwd), METHOD(tree_plan),
                         METHOD(tree_attn),      METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject *PyInit__paged_calls() { return PyModule_Create(&module); }
