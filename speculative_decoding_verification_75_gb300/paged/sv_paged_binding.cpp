// sv_paged_binding.cpp -- CPython module behind kv.py: checks the tensors of a
// call, fills the argument struct of include/sv_paged.h and calls the library.
//
// A call's host time is what short steps cost (a token for one request is a
// few microseconds of GPU time), and reading a tensor's properties from
// Python costs about a tenth of a microsecond each; here they are a few
// nanoseconds.  Shapes and types are checked here, sizes and alignments by
// the library.  Functions return the library's status; kv.py raises it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <string>

#include "sv_paged.h"

namespace {

struct Refused {
  PyObject *type;
  std::string text;
};

[[noreturn]] void type_error(const std::string &s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string &s) { throw Refused{PyExc_ValueError, s}; }

decltype(&sv_kv_write) fn_write;
decltype(&sv_kv_read) fn_read;
decltype(&sv_kv_compact) fn_compact;
decltype(&sv_tree_attention) fn_attn;
decltype(&sv_tree_attention_workspace_bytes) fn_ws;
decltype(&sv_kv_reserve) fn_reserve;
decltype(&sv_qk_norm_rope) fn_rope;

std::string str(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << ")";
  return o.str();
}

std::string dtype_name(at::ScalarType t) { return c10::toString(t); }

const at::Tensor *tensor_or_null(PyObject *o, const char *name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return &THPVariable_Unpack(o);
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  const at::Tensor *t = tensor_or_null(o, name);
  if (!t) type_error(std::string(name) + " must be a torch.Tensor");
  return *t;
}

// The device of a call: that of its first tensor.
int device_of(const at::Tensor &t, const char *name) {
  if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
  return t.get_device();
}

void on_device(const at::Tensor &t, const char *name, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    value_error(std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(dev));
}

void same(const at::Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType dtype, int dev) {
  if (t.scalar_type() != dtype)
    type_error(std::string(name) + " has dtype " + dtype_name(t.scalar_type()) + ", expected " + dtype_name(dtype));
  if (t.sizes() != shape)
    value_error(std::string(name) + " has shape " + str(t.sizes()) + ", expected " + str(shape));
  on_device(t, name, dev);
}

// An int32 tensor of this shape, contiguous; NULL for None.
const int32_t *ids(PyObject *o, const char *name, at::IntArrayRef shape, int dev, bool optional = false) {
  const at::Tensor *t = optional ? tensor_or_null(o, name) : &tensor(o, name);
  if (!t) return nullptr;
  same(*t, name, shape, at::kInt, dev);
  if (!t->is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return static_cast<const int32_t *>(t->data_ptr());
}

uint32_t *status_word(PyObject *o, int dev) {
  const at::Tensor *t = tensor_or_null(o, "status");
  if (!t) return nullptr;
  if (!t->is_cuda() || t->get_device() != dev || t->numel() != 1 ||
      (t->scalar_type() != at::kInt && t->scalar_type() != at::kUInt32))
    value_error("status must be a 1-element int32/uint32 tensor on the same device");
  return static_cast<uint32_t *>(t->data_ptr());
}

int code_of(at::ScalarType t) {
  return t == at::kBFloat16 ? SV_BF16 : t == at::kHalf ? SV_F16 : t == at::kFloat8_e4m3fn ? SV_E4M3
         : t == at::kByte ? SV_I4 : t == at::kFloat ? SV_F32 : -1;
}

// Caches of codes with scales, which take and are read by both 16-bit types.
bool scaled(int64_t code) { return code == SV_E4M3 || code == SV_I4; }

// Strides (layer, block) of a k / v pair whose last three dimensions are
// dense.  Dimensions of one element may have any stride.
void pool(const at::Tensor &k, const at::Tensor &v, const char *what, bool lead, int64_t &layer, int64_t &block) {
  const auto s = k.strides(), w = v.strides(), n = k.sizes();
  const int64_t d = k.dim();
  int64_t want = 1;
  for (int64_t i = d - 1; i >= d - 3; --i) {
    if (n[i] != 1 && s[i] != want) value_error(std::string(what) + ": the last three dimensions must be dense");
    want *= n[i];
  }
  for (int64_t i = 0; i < d; ++i)
    if (n[i] > 1 && s[i] != w[i]) value_error(std::string(what) + ": k and v must have the same strides");
  layer = lead ? s[0] : 0;
  block = s[lead ? 1 : 0];
}

// otab NULL: a call without block tables.
void take_cache(sv_kv_cache &c, PyObject *ok, PyObject *ov, PyObject *oks, PyObject *ovs, PyObject *otab, int dev,
                bool lead) {
  const at::Tensor &k = tensor(ok, "k_cache"), &v = tensor(ov, "v_cache");
  const int code = code_of(k.scalar_type());
  if (code < 0 || code == SV_F32) type_error("unsupported cache dtype " + dtype_name(k.scalar_type()));
  const auto n = k.sizes();
  const int64_t d = k.dim(), l = lead ? 1 : 0;
  if (d != 4 + l)
    value_error(std::string("k_cache and v_cache must be [num_blocks, kv heads, block size, head dim]") +
                (lead ? ", with the layers in front" : ""));
  on_device(k, "k_cache", dev);
  same(v, "v_cache", n, k.scalar_type(), dev);
  if (n[l + 1] == 0 || n[l + 2] == 0 || n[l + 3] == 0) value_error("k_cache has an empty dimension");
  pool(k, v, "k_cache and v_cache", lead, c.layer_stride, c.block_stride);
  const at::Tensor *ks = tensor_or_null(oks, "k_scale"), *vs = tensor_or_null(ovs, "v_scale");
  const int64_t per = code == SV_I4 ? 2 : 1;   // elements of an element of the tensor
  if (scaled(code)) {
    const std::string what = code == SV_I4 ? "a 4-bit" : "an e4m3";
    if (!ks || !vs) value_error(what + " cache needs k_scale and v_scale");
    if (n[l + 3] * per % SV_KV_GROUP) value_error("the head dim of " + what + " cache is a multiple of 32");
    c10::SmallVector<int64_t, 5> sn(n.begin(), n.end());
    sn.back() = sn.back() * per / SV_KV_GROUP;
    same(*ks, "k_scale", sn, at::kByte, dev);
    same(*vs, "v_scale", sn, at::kByte, dev);
    pool(*ks, *vs, "k_scale and v_scale", lead, c.scale_layer_stride, c.scale_block_stride);
    c.k_scale = static_cast<uint8_t *>(ks->data_ptr());
    c.v_scale = static_cast<uint8_t *>(vs->data_ptr());
  } else {
    if (ks || vs) value_error("k_scale and v_scale belong to a cache of codes (e4m3, 4 bits)");
  }
  if (otab) {
    const at::Tensor &tab = tensor(otab, "block_tables");
    if (tab.dim() != 2) value_error("block_tables must be [B, max_blocks]");
    c.block_tables = ids(otab, "block_tables", tab.sizes(), dev);
    c.max_blocks = tab.size(1);
  }
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.num_layers = lead ? n[0] : 1;
  c.num_blocks = n[l];
  c.num_kv_heads = n[l + 1];
  c.block_size = n[l + 2];
  c.head_dim = n[l + 3] * per;
  c.layer_stride *= per;
  c.block_stride *= per;
  c.dtype = code;
}

// Pointer and (b, t, head) strides of a [B, T, heads, D] tensor.
void *dense(const at::Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType dtype, int dev,
            int64_t (&s)[3]) {
  same(t, name, shape, dtype, dev);
  if (t.stride(3) != 1 && shape[3] != 1) value_error(std::string(name) + ": the last dimension must be dense");
  for (int i = 0; i < 3; ++i) s[i] = t.stride(i);
  return t.data_ptr();
}

// Refuses an output with two elements in one place (an expanded view).
void no_overlap(const at::Tensor &t, const char *name) {
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) > 1 && t.stride(i) == 0) value_error(std::string(name) + " must not be an expanded tensor");
}

// A tree mask [B, T, T] or [T, T], or None.
template <typename A>
void take_mask(A &a, PyObject *o, int dev) {
  const at::Tensor *m = tensor_or_null(o, "tree_mask");
  if (!m) return;
  if (m->scalar_type() != at::kBool) type_error("tree_mask must be a bool tensor");
  const int64_t d = m->dim();
  if ((d != 2 && d != 3) || m->size(d - 1) != a.T || m->size(d - 2) != a.T || (d == 3 && m->size(0) != a.B))
    value_error("tree_mask has shape " + str(m->sizes()) + ", expected " + str({a.T, a.T}) + " or " +
                str({a.B, a.T, a.T}));
  on_device(*m, "tree_mask", dev);
  if (a.T > 1 && (m->stride(d - 1) != 1 || m->stride(d - 2) != a.T))
    value_error("tree_mask: the last two dimensions must be dense");
  a.tree_mask = static_cast<const uint8_t *>(m->data_ptr());
  a.mask_batch_stride = d == 3 && a.B > 1 ? m->stride(0) : 0;
}

[[noreturn]] void not_together(const char *a, const at::Tensor &x, const at::Tensor &k, const at::Tensor &tab) {
  value_error(std::string(a) + " " + str(x.sizes()) + ", k_cache " + str(k.sizes()) + " and block_tables " +
              str(tab.sizes()) + " do not belong together");
}

// The call's stream: the current one of the device, or a raw handle.
struct Where {
  c10::cuda::OptionalCUDAGuard guard;
  std::optional<c10::cuda::CUDAStreamGuard> on;  // new tensors belong to the stream that uses them
  sv_stream_t stream;

  Where(PyObject *handle, int dev) {
    if (c10::cuda::current_device() != dev) guard.set_index(static_cast<c10::DeviceIndex>(dev));
    if (handle == Py_None) {
      stream = reinterpret_cast<sv_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
    } else {
      void *raw = PyLong_AsVoidPtr(handle);
      if (PyErr_Occurred()) throw Refused{nullptr, ""};
      stream = static_cast<sv_stream_t>(raw);
      on.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), static_cast<c10::DeviceIndex>(dev)));
    }
  }
};

template <typename F, typename A>
PyObject *call(F fn, const A &a, sv_stream_t stream) {
  sv_status rc;
  Py_BEGIN_ALLOW_THREADS
  rc = fn(&a, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, const F &f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused &r) {
    if (r.type) PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (key, value, k_cache, v_cache, block_tables, seq_lens, new_lens, k_scale, v_scale, status, stream)
PyObject *kv_write(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    sv_kv_write_args a = {};
    a.struct_bytes = sizeof a;
    const at::Tensor &key = tensor(o[0], "key"), &value = tensor(o[1], "value");
    const int dev = device_of(key, "key");
    take_cache(a.cache, o[2], o[3], o[7], o[8], o[4], dev, false);
    const at::Tensor &k = tensor(o[2], "k_cache"), &tab = tensor(o[4], "block_tables");
    if (key.dim() != 4) value_error("key must be [B, T, kv heads, head dim]");
    a.dtype = code_of(key.scalar_type());
    if (a.dtype != SV_BF16 && a.dtype != SV_F16) type_error("unsupported key dtype " + dtype_name(key.scalar_type()));
    if (!scaled(a.cache.dtype) && a.cache.dtype != a.dtype)
      type_error("a " + dtype_name(k.scalar_type()) + " cache takes no " + dtype_name(key.scalar_type()) + " keys");
    a.B = key.size(0);
    a.T = key.size(1);
    if (key.size(2) != a.cache.num_kv_heads || key.size(3) != a.cache.head_dim || tab.size(0) != a.B)
      not_together("key", key, k, tab);
    a.key = dense(key, "key", key.sizes(), key.scalar_type(), dev, a.key_stride);
    a.value = dense(value, "value", key.sizes(), key.scalar_type(), dev, a.value_stride);
    a.seq_lens = ids(o[5], "seq_lens", {a.B}, dev);
    a.new_lens = ids(o[6], "new_lens", {a.B}, dev, true);
    a.status = status_word(o[9], dev);
    const Where w(o[10], dev);
    return call(fn_write, a, w.stream);
  });
}

// (k_cache, v_cache, block_tables, lens, starts, out_k, out_v, k_scale, v_scale, status, stream)
PyObject *kv_read(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    sv_kv_read_args a = {};
    a.struct_bytes = sizeof a;
    const at::Tensor &k = tensor(o[0], "k_cache"), &tab = tensor(o[2], "block_tables");
    const int dev = device_of(k, "k_cache");
    take_cache(a.cache, o[0], o[1], o[7], o[8], o[2], dev, false);
    const at::Tensor &key = tensor(o[5], "out[0]"), &value = tensor(o[6], "out[1]");
    if (key.dim() != 4) value_error("out must be two [B, T, kv heads, head dim] tensors");
    a.dtype = code_of(key.scalar_type());
    if (a.dtype < 0 || scaled(a.dtype)) type_error("unsupported output dtype " + dtype_name(key.scalar_type()));
    a.B = tab.size(0);
    a.T = key.size(1);
    if (key.size(0) != a.B || key.size(2) != a.cache.num_kv_heads || key.size(3) != a.cache.head_dim)
      not_together("out", key, k, tab);
    a.key = dense(key, "out[0]", key.sizes(), key.scalar_type(), dev, a.key_stride);
    a.value = dense(value, "out[1]", key.sizes(), key.scalar_type(), dev, a.value_stride);
    no_overlap(key, "out[0]");
    no_overlap(value, "out[1]");
    a.lens = ids(o[3], "lens", {a.B}, dev);
    a.starts = ids(o[4], "starts", {a.B}, dev, true);
    a.status = status_word(o[9], dev);
    const Where w(o[10], dev);
    return call(fn_read, a, w.stream);
  });
}

// (path, num_accepted, seq_lens, block_tables, k_cache, v_cache, k_scale, v_scale, status, stream)
PyObject *kv_compact(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    sv_kv_compact_args a = {};
    a.struct_bytes = sizeof a;
    const at::Tensor &k = tensor(o[4], "k_cache"), &tab = tensor(o[3], "block_tables");
    const int dev = device_of(k, "k_cache");
    take_cache(a.cache, o[4], o[5], o[6], o[7], o[3], dev, k.dim() == 5);
    const at::Tensor &path = tensor(o[0], "path");
    if (path.dim() != 2) value_error("path must be [B, P]");
    a.B = tab.size(0);
    a.P = path.size(1);
    a.path = ids(o[0], "path", {a.B, a.P}, dev);
    a.num_accepted = ids(o[1], "num_accepted", {a.B}, dev);
    a.seq_lens = ids(o[2], "seq_lens", {a.B}, dev);
    a.status = status_word(o[8], dev);
    const Where w(o[9], dev);
    return call(fn_compact, a, w.stream);
  });
}

// A tuple of new references; NULL where one of them is.
PyObject *tuple_of(std::initializer_list<PyObject *> items) {
  PyObject *t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  bool whole = t != nullptr;
  for (PyObject *x : items) whole = whole && x;
  for (PyObject *x : items) {
    if (whole) PyTuple_SET_ITEM(t, i++, x);
    else Py_XDECREF(x);
  }
  if (!whole) Py_CLEAR(t);
  return t;
}

PyObject *given_or(PyObject *given, const at::Tensor &made) {
  if (given == Py_None) return THPVariable_Wrap(made);
  Py_INCREF(given);
  return given;
}

// (query, k_cache, v_cache, block_tables, seq_lens, tree_mask, new_lens, scale, k_scale, v_scale, out, lse,
//  workspace, status, stream) -> (status, out)
PyObject *tree_attention(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject * {
    sv_tree_attention_args a = {};
    a.struct_bytes = sizeof a;
    const at::Tensor &q = tensor(o[0], "query");
    const int dev = device_of(q, "query");
    take_cache(a.cache, o[1], o[2], o[8], o[9], o[3], dev, false);
    const at::Tensor &k = tensor(o[1], "k_cache"), &tab = tensor(o[3], "block_tables");
    if (q.dim() != 4) value_error("query must be [B, T, heads, head dim]");
    a.dtype = code_of(q.scalar_type());
    if (a.dtype != SV_BF16 && a.dtype != SV_F16) type_error("unsupported query dtype " + dtype_name(q.scalar_type()));
    if (!scaled(a.cache.dtype) && a.cache.dtype != a.dtype)
      type_error(dtype_name(q.scalar_type()) + " queries do not read a " + dtype_name(k.scalar_type()) + " cache");
    a.B = q.size(0);
    a.T = q.size(1);
    a.num_heads = q.size(2);
    if (q.size(3) != a.cache.head_dim || a.num_heads % a.cache.num_kv_heads || tab.size(0) != a.B)
      not_together("query", q, k, tab);
    a.query = dense(q, "query", q.sizes(), q.scalar_type(), dev, a.query_stride);
    a.seq_lens = ids(o[4], "seq_lens", {a.B}, dev);
    a.new_lens = ids(o[6], "new_lens", {a.B}, dev, true);
    take_mask(a, o[5], dev);
    if (o[7] == Py_None) {
      a.scale = 1.0 / std::sqrt(static_cast<double>(a.cache.head_dim));
    } else {
      a.scale = PyFloat_AsDouble(o[7]);
      if (PyErr_Occurred()) throw Refused{nullptr, ""};
    }
    const at::Tensor *out = tensor_or_null(o[10], "out");
    if (out) {
      same(*out, "out", q.sizes(), q.scalar_type(), dev);
      if (!out->is_contiguous()) value_error("out must be contiguous");
    }
    if (const at::Tensor *l = tensor_or_null(o[11], "lse")) {
      same(*l, "lse", {a.B, a.T, a.num_heads}, at::kFloat, dev);
      if (!l->is_contiguous()) value_error("lse must be contiguous");
      a.lse = static_cast<float *>(l->data_ptr());
    }
    const at::Tensor *ws = tensor_or_null(o[12], "workspace");
    if (ws) {
      same(*ws, "workspace", ws->sizes(), at::kByte, dev);
      if (!ws->is_contiguous()) value_error("workspace must be contiguous");
    }
    a.status = status_word(o[13], dev);
    const Where w(o[14], dev);
    at::Tensor new_out, new_ws;
    if (!out) {
      new_out = at::empty(q.sizes(), q.options().memory_format(at::MemoryFormat::Contiguous));
      out = &new_out;
    }
    if (!ws) {
      const size_t need = fn_ws(a.B, a.T, a.num_heads, a.cache.num_kv_heads, a.cache.head_dim);
      new_ws = at::empty({static_cast<int64_t>(need ? need : 256)}, q.options().dtype(at::kByte));
      ws = &new_ws;
    }
    a.out = out->data_ptr();
    a.workspace = ws->data_ptr();
    a.workspace_bytes = static_cast<uint64_t>(ws->numel());
    PyObject *rc = call(fn_attn, a, w.stream);
    if (!rc) return nullptr;
    return tuple_of({rc, given_or(o[10], new_out)});
  });
}

// A result of this shape: the given tensor, contiguous, or a new one.
template <typename E>
E *result(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dtype, const at::TensorOptions &like,
          int dev, at::Tensor &made) {
  const at::Tensor *t = tensor_or_null(o, name);
  if (t) {
    same(*t, name, shape, dtype, dev);
    if (!t->is_contiguous()) value_error(std::string(name) + " must be contiguous");
  } else {
    made = at::empty(shape, like.dtype(dtype));
    t = &made;
  }
  return static_cast<E *>(t->data_ptr());
}

// (seq_lens, new_lens, block_tables, block_size, free_list, free_count, tree_mask, max_new, slots, positions,
//  reserved, status, stream) -> (status, slots, positions, reserved)
PyObject *kv_reserve(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    sv_kv_reserve_args a = {};
    a.struct_bytes = sizeof a;
    const at::Tensor &seq = tensor(o[0], "seq_lens"), &tab = tensor(o[2], "block_tables");
    const int dev = device_of(seq, "seq_lens");
    if (tab.dim() != 2) value_error("block_tables must be [B, max_blocks]");
    a.B = tab.size(0);
    a.max_blocks = tab.size(1);
    a.seq_lens = ids(o[0], "seq_lens", {a.B}, dev);
    a.new_lens = ids(o[1], "new_lens", {a.B}, dev, true);
    a.block_tables = const_cast<int32_t *>(ids(o[2], "block_tables", tab.sizes(), dev));
    a.block_size = PyLong_AsLongLong(o[3]);
    if (PyErr_Occurred()) throw Refused{nullptr, ""};
    const at::Tensor &list = tensor(o[4], "free_list");
    if (list.dim() != 1) value_error("free_list must have 1 dimension");
    a.free_list = ids(o[4], "free_list", list.sizes(), dev);
    a.free_capacity = list.numel();
    const at::Tensor &cnt = tensor(o[5], "free_count");
    if (cnt.numel() != 1) value_error("free_count must have 1 element");
    a.free_count = const_cast<int32_t *>(ids(o[5], "free_count", cnt.sizes(), dev));
    // T: said, or that of the first tensor which has it.
    if (o[7] != Py_None) {
      a.T = PyLong_AsLongLong(o[7]);
      if (PyErr_Occurred()) throw Refused{nullptr, ""};
      if (a.T < 0) value_error("max_new is negative");
    } else {
      const at::Tensor *m = tensor_or_null(o[6], "tree_mask");
      const at::Tensor *s = tensor_or_null(o[8], "slots");
      if (s && s->dim() == 2) a.T = s->size(1);
      else if (m && m->dim() >= 2) a.T = m->size(m->dim() - 1);
      else value_error("max_new is needed when neither slots nor tree_mask says how many new tokens there are");
    }
    take_mask(a, o[6], dev);
    a.status = status_word(o[11], dev);
    const Where w(o[12], dev);
    at::Tensor slots, positions, reserved;
    const auto like = seq.options();
    a.slots = result<int64_t>(o[8], "slots", {a.B, a.T}, at::kLong, like, dev, slots);
    a.positions = result<int32_t>(o[9], "positions", {a.B, a.T}, at::kInt, like, dev, positions);
    a.reserved = result<int32_t>(o[10], "reserved", {a.B}, at::kInt, like, dev, reserved);
    PyObject *rc = call(fn_reserve, a, w.stream);
    if (!rc) return nullptr;
    return tuple_of({rc, given_or(o[8], slots), given_or(o[9], positions), given_or(o[10], reserved)});
  });
}

// (query, key, cos_sin, positions, q_weight, k_weight, eps, interleaved, out, key_out, value, k_cache, v_cache, slots,
//  k_scale, v_scale, status, stream) -> (status, out, key_out or None)
PyObject *qk_norm_rope(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return guarded(n, 18, [&]() -> PyObject * {
    sv_qk_norm_rope_args a = {};
    a.struct_bytes = sizeof a;
    const at::Tensor &q = tensor(o[0], "query"), &k = tensor(o[1], "key");
    const int dev = device_of(q, "query");
    if (q.dim() != 4) value_error("query must be [B, T, heads, head dim]");
    if (k.dim() != 4 || k.size(0) != q.size(0) || k.size(1) != q.size(1) || k.size(3) != q.size(3))
      value_error("query " + str(q.sizes()) + " and key " + str(k.sizes()) + " do not belong together");
    a.dtype = code_of(q.scalar_type());
    if (a.dtype != SV_BF16 && a.dtype != SV_F16) type_error("unsupported query dtype " + dtype_name(q.scalar_type()));
    a.B = q.size(0);
    a.T = q.size(1);
    a.num_heads = q.size(2);
    a.num_kv_heads = k.size(2);
    a.head_dim = q.size(3);
    a.query = dense(q, "query", q.sizes(), q.scalar_type(), dev, a.query_stride);
    a.key = dense(k, "key", k.sizes(), q.scalar_type(), dev, a.key_stride);
    const at::Tensor &cs = tensor(o[2], "cos_sin");
    if (cs.dim() != 2) value_error("cos_sin must be [positions, rotary dim]");
    same(cs, "cos_sin", cs.sizes(), at::kFloat, dev);
    if (!cs.is_contiguous()) value_error("cos_sin must be contiguous");
    a.cos_sin = static_cast<const float *>(cs.data_ptr());
    a.num_positions = cs.size(0);
    a.rotary_dim = cs.size(1);
    a.positions = ids(o[3], "positions", {a.B, a.T}, dev);
    const auto weight = [&](PyObject *x, const char *name) -> const void * {
      const at::Tensor *t = tensor_or_null(x, name);
      if (!t) return nullptr;
      same(*t, name, {a.head_dim}, q.scalar_type(), dev);
      if (!t->is_contiguous()) value_error(std::string(name) + " must be contiguous");
      return t->data_ptr();
    };
    a.q_weight = weight(o[4], "q_weight");
    a.k_weight = weight(o[5], "k_weight");
    a.eps = PyFloat_AsDouble(o[6]);
    if (PyErr_Occurred()) throw Refused{nullptr, ""};
    const int pairs = PyObject_IsTrue(o[7]);
    if (pairs < 0) throw Refused{nullptr, ""};
    a.interleaved = pairs;
    const bool cached = o[11] != Py_None || o[12] != Py_None;
    if (cached) {
      take_cache(a.cache, o[11], o[12], o[14], o[15], nullptr, dev, false);
      const at::Tensor &kc = tensor(o[11], "k_cache");
      if (!scaled(a.cache.dtype) && a.cache.dtype != a.dtype)
        type_error("a " + dtype_name(kc.scalar_type()) + " cache takes no " + dtype_name(k.scalar_type()) + " keys");
      if (a.cache.num_kv_heads != a.num_kv_heads || a.cache.head_dim != a.head_dim)
        value_error("key " + str(k.sizes()) + " and k_cache " + str(kc.sizes()) + " do not belong together");
      const at::Tensor &v = tensor(o[10], "value"), &s = tensor(o[13], "slots");
      a.value = dense(v, "value", k.sizes(), q.scalar_type(), dev, a.value_stride);
      same(s, "slots", {a.B, a.T}, at::kLong, dev);
      if (!s.is_contiguous()) value_error("slots must be contiguous");
      a.slots = static_cast<const int64_t *>(s.data_ptr());
    } else {
      if (o[10] != Py_None || o[13] != Py_None || o[14] != Py_None || o[15] != Py_None)
        value_error("value, slots and scales belong to k_cache and v_cache");
    }
    a.status = status_word(o[16], dev);
    const at::Tensor *out = tensor_or_null(o[8], "out"), *ko = tensor_or_null(o[9], "key_out");
    if (out) {
      a.out = dense(*out, "out", q.sizes(), q.scalar_type(), dev, a.out_stride);
      no_overlap(*out, "out");
    }
    if (ko) {
      a.key_out = dense(*ko, "key_out", k.sizes(), q.scalar_type(), dev, a.key_out_stride);
      no_overlap(*ko, "key_out");
    }
    const Where w(o[17], dev);
    at::Tensor new_out, new_ko;
    const auto like = q.options().memory_format(at::MemoryFormat::Contiguous);
    if (!out) {
      new_out = at::empty(q.sizes(), like);
      a.out = dense(new_out, "out", q.sizes(), q.scalar_type(), dev, a.out_stride);
    }
    if (!ko && !cached) {
      new_ko = at::empty(k.sizes(), like);
      a.key_out = dense(new_ko, "key_out", k.sizes(), q.scalar_type(), dev, a.key_out_stride);
    }
    // An empty slots tensor has no address; its call has nothing to do.
    if (a.B == 0 || a.T == 0) return tuple_of({PyLong_FromLong(SV_OK), given_or(o[8], new_out),
                                              !ko && cached ? Py_NewRef(Py_None) : given_or(o[9], new_ko)});
    PyObject *rc = call(fn_rope, a, w.stream);
    if (!rc) return nullptr;
    return tuple_of({rc, given_or(o[8], new_out), !ko && cached ? Py_NewRef(Py_None) : given_or(o[9], new_ko)});
  });
}

// (path of the library)
PyObject *bind_library(PyObject *, PyObject *arg) {
  const char *path = PyUnicode_AsUTF8(arg);
  if (!path) return nullptr;
  void *lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_SetString(PyExc_OSError, dlerror());
    return nullptr;
  }
  fn_write = reinterpret_cast<decltype(fn_write)>(dlsym(lib, "sv_kv_write"));
  fn_read = reinterpret_cast<decltype(fn_read)>(dlsym(lib, "sv_kv_read"));
  fn_compact = reinterpret_cast<decltype(fn_compact)>(dlsym(lib, "sv_kv_compact"));
  fn_attn = reinterpret_cast<decltype(fn_attn)>(dlsym(lib, "sv_tree_attention"));
  fn_ws = reinterpret_cast<decltype(fn_ws)>(dlsym(lib, "sv_tree_attention_workspace_bytes"));
  fn_reserve = reinterpret_cast<decltype(fn_reserve)>(dlsym(lib, "sv_kv_reserve"));
  fn_rope = reinterpret_cast<decltype(fn_rope)>(dlsym(lib, "sv_qk_norm_rope"));
  if (!fn_write || !fn_read || !fn_compact || !fn_attn || !fn_ws || !fn_reserve || !fn_rope) {
    PyErr_SetString(PyExc_OSError, "the library lacks the paged-cache entry points");
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"kv_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv_write)), METH_FASTCALL, nullptr},
    {"kv_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv_read)), METH_FASTCALL, nullptr},
    {"kv_compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv_compact)), METH_FASTCALL, nullptr},
    {"tree_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(tree_attention)), METH_FASTCALL, nullptr},
    {"kv_reserve", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv_reserve)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"bind_library", bind_library, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_svkv", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__svkv(void) { return PyModule_Create(&module); }
