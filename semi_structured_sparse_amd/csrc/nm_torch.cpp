// The quick way from torch tensors to the calls of nm_decode.h and nm_block.h: a Python extension
// that checks the arguments as decode.py and block.py do, makes the outputs and calls the library, in 3 to 6 us of the
// host where decode.py alone takes 9 to 16, launch and outputs' allocation included (4 is what
// torch takes to fill an empty tensor; a decoding step makes three such calls a layer). Each
// function returns NotImplemented where anything is not as it should be (a check that fails, a
// tensor on another device than the current one, memory that runs out, a call that the library
// refuses); the Python module then goes its own way, whose checks say what it is. Nothing here touches
// tensor data.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <cmath>
#include <cstring>

#include "nm_block.h"
#include "nm_decode.h"

namespace {

struct Library {
  decltype(&nm_rope) rope;
  decltype(&nm_kv_append) kv_append;
  decltype(&nm_rope_kv_append) rope_kv_append;
  decltype(&nm_kv_read) kv_read;
  decltype(&nm_kv_compact) kv_compact;
  decltype(&nm_tree_attention) tree_attention;
  decltype(&nm_verify_chain) verify_chain;
  decltype(&nm_verify_tree) verify_tree;
  decltype(&nm_linear) linear;
  decltype(&nm_gated) gated;
  decltype(&nm_norm) norm;
  decltype(&nm_block_norm) block_norm;
  decltype(&nm_logprobs) logprobs;
};
Library lib;   // the addresses of the library decode.py loaded

// What the checks found out; a call's arguments are good if every one was.
struct Call {
  bool good = true;
  int device = -1;
  void* stream = nullptr;

  // The first tensor names the device, which has to be the current one.
  const at::Tensor* first(PyObject* o) {
    if (!THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != c10::hip::current_device()) return fail();
    device = int(t.get_device());
    stream = c10::hip::getCurrentHIPStream(c10::DeviceIndex(device)).stream();
    return &t;
  }
  const at::Tensor* fail() {
    good = false;
    return nullptr;
  }
  const at::Tensor* tensor(PyObject* o, at::ScalarType type) {
    if (!good || !THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != device) return fail();
    return &t;
  }
  // A contiguous tensor of a shape; None gives NULL where that is allowed.
  template <class T>
  T* plain(PyObject* o, at::ScalarType type, at::IntArrayRef shape, bool none = false) {
    if (none && o == Py_None) return nullptr;
    const at::Tensor* t = tensor(o, type);
    if (t == nullptr || t->sizes() != shape || !t->is_contiguous()) {
      good = false;
      return nullptr;
    }
    return static_cast<T*>(t->data_ptr());
  }
  // fp16 [..., heads, head_dim] with contiguous heads and evenly spaced tokens; its token stride.
  uint16_t* rows(PyObject* o, int64_t dims, int64_t* stride) {
    const at::Tensor* t = tensor(o, at::kHalf);
    if (t == nullptr || t->dim() != dims) return static_cast<uint16_t*>(bad());
    const auto size = t->sizes(), step = t->strides();
    const int64_t row = size[dims - 1] * size[dims - 2];
    if ((step[dims - 1] != 1 && size[dims - 1] > 1) || (step[dims - 2] != size[dims - 1] && size[dims - 2] > 1))
      return static_cast<uint16_t*>(bad());
    if (dims == 3 || size[1] == 1)
      *stride = size[0] > 1 ? step[0] : row;
    else if (size[0] > 1 && step[0] != size[1] * step[1])
      return static_cast<uint16_t*>(bad());
    else
      *stride = step[1];
    return static_cast<uint16_t*>(t->data_ptr());
  }
  void* bad() {
    good = false;
    return nullptr;
  }
  double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      good = false;
    }
    return v;
  }
  int64_t whole(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      good = false;
    }
    return v;
  }
  // A cache's four tensors, from a[0] on.
  nm_kv_cache cache(PyObject* const* a) {
    nm_kv_cache c{};
    if (!good || !THPVariable_Check(a[0])) {
      good = false;
      return c;
    }
    const at::Tensor& k = THPVariable_Unpack(a[0]);
    const auto type = k.scalar_type();
    c.format = type == at::kHalf ? NM_KV_FP16 : type == at::kChar ? NM_KV_INT8 : type == at::kFloat8_e4m3fn ? NM_KV_E4M3 : -1;
    if (c.format < 0 || k.dim() != 4) {
      good = false;
      return c;
    }
    const auto shape = k.sizes();
    c.k = plain<void>(a[0], type, shape);
    c.v = plain<void>(a[1], type, shape);
    if (c.format != NM_KV_FP16) {
      c.k_scale = plain<float>(a[2], at::kFloat, shape.slice(0, 3));
      c.v_scale = plain<float>(a[3], at::kFloat, shape.slice(0, 3));
    }
    if (shape[1] > INT32_MAX || shape[2] > INT32_MAX || shape[3] > INT32_MAX) good = false;
    c.blocks = shape[0];
    c.kv_heads = int32_t(shape[1]);
    c.page = int32_t(shape[2]);
    c.head_dim = int32_t(shape[3]);
    return c;
  }
  // A page table's width, and the address of it.
  int32_t* table(PyObject* o, int64_t batch, int64_t* width) {
    const at::Tensor* t = tensor(o, at::kInt);
    if (t == nullptr || t->dim() != 2 || t->size(0) != batch || !t->is_contiguous()) {
      good = false;
      return nullptr;
    }
    *width = t->size(1);
    return static_cast<int32_t*>(t->data_ptr());
  }
  double* turns(PyObject* o, int* rot) {
    const at::Tensor* t = tensor(o, at::kDouble);
    if (t == nullptr || t->dim() != 1 || !t->is_contiguous() || t->size(0) > 512) {
      good = false;
      return nullptr;
    }
    *rot = int(2 * t->size(0));
    return static_cast<double*>(t->data_ptr());
  }
};

PyObject* not_here() { Py_RETURN_NOTIMPLEMENTED; }

at::Tensor made(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, c10::DeviceIndex(device)));
}

// A given output, or a new one.
THPObjectPtr output(PyObject* given, at::IntArrayRef shape, int device) {
  if (given == Py_None) return THPObjectPtr(THPVariable_Wrap(made(shape, at::kHalf, device)));
  Py_INCREF(given);
  return THPObjectPtr(given);
}

bool same_shape(PyObject* o, const at::Tensor& t) {
  return o == Py_None || (THPVariable_Check(o) && THPVariable_Unpack(o).sizes() == t.sizes());
}

// Ends a call: the result where the library took it.
PyObject* finish(int status, THPObjectPtr result) { return status == 0 ? result.release() : not_here(); }

THPObjectPtr none() {
  Py_INCREF(Py_None);
  return THPObjectPtr(Py_None);
}

// (x, positions, turns, layout, scale, out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  const at::Tensor* x = n == 6 ? c.first(a[0]) : nullptr;
  if (x == nullptr || x->dim() != 3 || !same_shape(a[5], *x)) return not_here();
  int64_t xs = 0, ys = 0;
  int rot = 0;
  uint16_t* xp = c.rows(a[0], 3, &xs);
  const int64_t tokens = x->size(0), heads = x->size(1), dim = x->size(2);
  auto* positions = c.plain<int32_t>(a[1], at::kInt, {tokens});
  double* turns = c.turns(a[2], &rot);
  const int layout = int(c.whole(a[3]));
  const float scale = float(c.number(a[4]));
  if (!c.good || dim > 1024) return not_here();
  THPObjectPtr out = output(a[5], x->sizes(), c.device);
  uint16_t* yp = c.rows(out, 3, &ys);
  if (!c.good) return not_here();
  return finish(lib.rope(xp, yp, positions, turns, tokens, heads, int(dim), rot, layout, scale, xs, ys, c.stream),
                std::move(out));
}

// (cache x 4, k, v, table, start, count)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  const at::Tensor* k = n == 9 ? c.first(a[4]) : nullptr;
  if (k == nullptr || k->dim() != 4 || a[5] == Py_None || !same_shape(a[5], *k)) return not_here();
  const nm_kv_cache cache = c.cache(a);
  int64_t ks = 0, vs = 0, width = 0;
  uint16_t *kp = c.rows(a[4], 4, &ks), *vp = c.rows(a[5], 4, &vs);
  const int64_t batch = k->size(0), tokens = k->size(1);
  int32_t* table = c.table(a[6], batch, &width);
  auto* start = c.plain<int32_t>(a[7], at::kInt, {batch});
  auto* count = c.plain<int32_t>(a[8], at::kInt, {batch}, true);
  if (!c.good || k->size(2) != cache.kv_heads || k->size(3) != cache.head_dim) return not_here();
  return finish(lib.kv_append(&cache, kp, vp, ks, vs, table, width, start, count, batch, tokens, c.stream), none());
}

// (cache x 4, q, k, v, positions, turns, table, start, count, layout, scale, out)
PyObject* rope_kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  const at::Tensor* k = n == 15 ? c.first(a[5]) : nullptr;
  if (k == nullptr || k->dim() != 4 || a[6] == Py_None || !same_shape(a[6], *k)) return not_here();
  const nm_kv_cache cache = c.cache(a);
  int64_t qs = 0, os = 0, ks = 0, vs = 0, width = 0, heads = 0;
  int rot = 0;
  uint16_t *kp = c.rows(a[5], 4, &ks), *vp = c.rows(a[6], 4, &vs), *qp = nullptr, *op = nullptr;
  const int64_t batch = k->size(0), tokens = k->size(1);
  auto* positions = c.plain<int32_t>(a[7], at::kInt, {batch, tokens});
  double* turns = c.turns(a[8], &rot);
  int32_t* table = c.table(a[9], batch, &width);
  auto* start = c.plain<int32_t>(a[10], at::kInt, {batch});
  auto* count = c.plain<int32_t>(a[11], at::kInt, {batch}, true);
  if (!c.good || k->size(2) != cache.kv_heads || k->size(3) != cache.head_dim) return not_here();
  const int layout = int(c.whole(a[12]));
  const float scale = float(c.number(a[13]));
  THPObjectPtr out = none();
  if (a[4] != Py_None) {
    qp = c.rows(a[4], 4, &qs);
    if (!c.good) return not_here();
    const at::Tensor& q = THPVariable_Unpack(a[4]);
    heads = q.size(2);
    if (q.size(0) != batch || q.size(1) != tokens || q.size(3) != cache.head_dim || !same_shape(a[14], q)) return not_here();
    out = output(a[14], q.sizes(), c.device);
    op = c.rows(out, 4, &os);
  }
  if (!c.good) return not_here();
  return finish(lib.rope_kv_append(&cache, qp, op, heads, qs, os, kp, vp, ks, vs, positions, turns, rot, layout, scale,
                                   table, width, start, count, batch, tokens, c.stream),
                std::move(out));
}

// (cache x 4, table, start, tokens, count, k_out, v_out)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  const at::Tensor* t = n == 10 ? c.first(a[4]) : nullptr;
  if (t == nullptr || t->dim() != 2) return not_here();
  const nm_kv_cache cache = c.cache(a);
  const int64_t batch = t->size(0), tokens = c.whole(a[6]);
  int64_t width = 0;
  int32_t* table = c.table(a[4], batch, &width);
  auto* start = c.plain<int32_t>(a[5], at::kInt, {batch});
  auto* count = c.plain<int32_t>(a[7], at::kInt, {batch}, true);
  if (!c.good || tokens < 1 || tokens > (int64_t(1) << 24)) return not_here();
  const int64_t shape[4] = {batch, tokens, cache.kv_heads, cache.head_dim};
  THPObjectPtr k = output(a[8], shape, c.device), v = output(a[9], shape, c.device);
  auto *kp = c.plain<uint16_t>(k, at::kHalf, shape), *vp = c.plain<uint16_t>(v, at::kHalf, shape);
  if (!c.good) return not_here();
  return finish(lib.kv_read(&cache, kp, vp, table, width, start, count, batch, tokens, c.stream),
                THPObjectPtr(PyTuple_Pack(2, k.get(), v.get())));
}

// (cache x 4, table, start, path, accepted)
PyObject* kv_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  const at::Tensor* t = n == 8 ? c.first(a[4]) : nullptr;
  const at::Tensor* p = c.good && t != nullptr ? c.tensor(a[6], at::kInt) : nullptr;
  if (p == nullptr || t->dim() != 2 || p->dim() != 2) return not_here();
  const nm_kv_cache cache = c.cache(a);
  const int64_t batch = t->size(0), nodes = p->size(1);
  int64_t width = 0;
  int32_t* table = c.table(a[4], batch, &width);
  auto* start = c.plain<int32_t>(a[5], at::kInt, {batch});
  auto* path = c.plain<int32_t>(a[6], at::kInt, {batch, nodes});
  auto* accepted = c.plain<int32_t>(a[7], at::kInt, {batch});
  if (!c.good) return not_here();
  return finish(lib.kv_compact(&cache, table, width, start, path, accepted, batch, nodes, c.stream), none());
}

// A workspace's address and bytes; None: none.
char* workspace(Call& c, PyObject* o, size_t* bytes) {
  *bytes = 0;
  if (o == Py_None) return nullptr;
  const at::Tensor* t = c.tensor(o, at::kByte);
  if (t == nullptr || t->dim() != 1 || !t->is_contiguous()) return static_cast<char*>(c.bad());
  *bytes = size_t(t->numel());
  return static_cast<char*>(t->data_ptr());
}

// (q, cache x 4, table, context, mask, count, scale, workspace, out)
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  const at::Tensor* q = n == 12 ? c.first(a[0]) : nullptr;
  if (q == nullptr || q->dim() != 4) return not_here();
  const nm_kv_cache cache = c.cache(a + 1);
  int64_t qs = 0, width = 0;
  uint16_t* qp = c.rows(a[0], 4, &qs);
  const int64_t batch = q->size(0), tokens = q->size(1), heads = q->size(2);
  int32_t* table = c.table(a[5], batch, &width);
  auto* context = c.plain<int32_t>(a[6], at::kInt, {batch});
  auto* mask = c.plain<uint64_t>(a[7], at::kLong, {batch, tokens}, true);
  auto* count = c.plain<int32_t>(a[8], at::kInt, {batch}, true);
  size_t bytes = 0;
  char* ws = workspace(c, a[10], &bytes);
  const float scale = a[9] == Py_None ? float(1.0 / std::sqrt(double(cache.head_dim))) : float(c.number(a[9]));
  if (!c.good || q->size(3) != cache.head_dim) return not_here();
  THPObjectPtr out = output(a[11], q->sizes(), c.device);
  auto* op = c.plain<uint16_t>(out, at::kHalf, q->sizes());
  if (!c.good) return not_here();
  return finish(lib.tree_attention(&cache, qp, op, heads, qs, table, width, context, mask, count, batch, tokens, scale, ws,
                                   bytes, c.stream),
                std::move(out));
}

// (target, draft or parents, tokens, uniforms, count, workspace); parents: a tree's.
PyObject* verify(PyObject* const* a, Py_ssize_t n, bool tree) {
  Call c;
  const at::Tensor* t = n == 6 ? c.first(a[0]) : nullptr;
  if (t == nullptr || t->dim() != 3) return not_here();
  const int64_t batch = t->size(0), nodes = t->size(1), vocab = t->size(2);
  auto* target = c.plain<float>(a[0], at::kFloat, t->sizes());
  auto* draft = tree ? nullptr : c.plain<float>(a[1], at::kFloat, {batch, nodes - 1, vocab}, true);
  auto* parents = tree ? c.plain<int32_t>(a[1], at::kInt, {batch, nodes}) : nullptr;
  auto* tokens = c.plain<int32_t>(a[2], at::kInt, {batch, nodes});
  auto* uniforms = c.plain<float>(a[3], at::kFloat, {batch, nodes});
  auto* count = c.plain<int32_t>(a[4], at::kInt, {batch}, true);
  size_t bytes = 0;
  char* ws = workspace(c, a[5], &bytes);
  if (!c.good) return not_here();
  const at::Tensor accepted = made({batch}, at::kInt, c.device), out = made({batch, nodes}, at::kInt, c.device);
  auto *ap = static_cast<int32_t*>(accepted.data_ptr()), *op = static_cast<int32_t*>(out.data_ptr());
  if (!tree) {
    if (lib.verify_chain(target, draft, tokens, uniforms, count, ap, op, batch, nodes, vocab, ws, bytes, c.stream) != 0)
      return not_here();
    return Py_BuildValue("(NN)", THPVariable_Wrap(accepted), THPVariable_Wrap(out));
  }
  const at::Tensor path = made({batch, nodes}, at::kInt, c.device);
  if (lib.verify_tree(target, tokens, parents, uniforms, count, ap, op, static_cast<int32_t*>(path.data_ptr()), batch, nodes,
                      vocab, ws, bytes, c.stream) != 0)
    return not_here();
  return Py_BuildValue("(NNN)", THPVariable_Wrap(accepted), THPVariable_Wrap(out), THPVariable_Wrap(path));
}
PyObject* verify_chain(PyObject*, PyObject* const* a, Py_ssize_t n) { return verify(a, n, false); }
PyObject* verify_tree(PyObject*, PyObject* const* a, Py_ssize_t n) { return verify(a, n, true); }

// A packed matrix of rows x cols and pattern N:M: values a[0], masks a[1].
struct Packed {
  uint16_t* values;
  uint32_t* masks;
  int64_t rows, cols;
};
Packed packed(Call& c, PyObject* const* a, int64_t N, int64_t M) {
  Packed p{};
  const at::Tensor* m = c.tensor(a[1], at::kInt);
  if (m == nullptr || m->dim() != 2 || !m->is_contiguous() || N < 1 || N > 32 || M < 1 || M > 32 || m->size(1) > (int64_t(1) << 26)) {
    c.good = false;
    return p;
  }
  p.rows = m->size(0);
  p.cols = 32 * m->size(1);
  p.masks = static_cast<uint32_t*>(m->data_ptr());
  p.values = c.plain<uint16_t>(a[0], at::kHalf, {p.rows, p.cols * N / M});
  return p;
}

// X fp16 [cols] or [batch, cols] and the output of its products with `rows` rows.
struct Vectors {
  uint16_t* x = nullptr;
  int64_t batch = 1;
  c10::SmallVector<int64_t, 2> out_shape;
};
Vectors vectors(Call& c, PyObject* o, const Packed& w) {
  Vectors v;
  const at::Tensor* x = c.tensor(o, at::kHalf);
  if (x == nullptr || (x->dim() != 1 && x->dim() != 2) || x->size(-1) != w.cols || !x->is_contiguous()) {
    c.good = false;
    return v;
  }
  v.x = static_cast<uint16_t*>(x->data_ptr());
  if (x->dim() == 2) v.out_shape.push_back(v.batch = x->size(0));
  v.out_shape.push_back(w.rows);
  return v;
}

// (values, masks, X, N, M, bias, activation, scale, residual, workspace, out)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  if (n != 11 || c.first(a[2]) == nullptr) return not_here();
  const int64_t N = c.whole(a[3]), M = c.whole(a[4]);
  const Packed w = packed(c, a, N, M);
  if (!c.good) return not_here();
  const Vectors v = vectors(c, a[2], w);
  auto* bias = c.plain<uint16_t>(a[5], at::kHalf, {w.rows}, true);
  auto* residual = c.plain<uint16_t>(a[8], at::kHalf, v.out_shape, true);
  const int activation = int(c.whole(a[6]));
  const float scale = float(c.number(a[7]));
  size_t bytes = 0;
  char* ws = workspace(c, a[9], &bytes);
  if (!c.good) return not_here();
  THPObjectPtr out = output(a[10], v.out_shape, c.device);
  auto* op = c.plain<uint16_t>(out, at::kHalf, v.out_shape);
  if (!c.good) return not_here();
  return finish(lib.linear(w.values, w.masks, v.x, op, w.rows, w.cols, v.batch, int(N), int(M), bias, activation, scale,
                           residual, ws, bytes, c.stream),
                std::move(out));
}

// (gate values, gate masks, up values, up masks, X, N, M, activation, gate_bias, up_bias, workspace, out)
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  if (n != 12 || c.first(a[4]) == nullptr) return not_here();
  const int64_t N = c.whole(a[5]), M = c.whole(a[6]);
  const Packed g = packed(c, a, N, M), u = packed(c, a + 2, N, M);
  if (!c.good || g.rows != u.rows || g.cols != u.cols) return not_here();
  const Vectors v = vectors(c, a[4], g);
  const int activation = int(c.whole(a[7]));
  auto* gate_bias = c.plain<uint16_t>(a[8], at::kHalf, {g.rows}, true);
  auto* up_bias = c.plain<uint16_t>(a[9], at::kHalf, {g.rows}, true);
  size_t bytes = 0;
  char* ws = workspace(c, a[10], &bytes);
  if (!c.good) return not_here();
  THPObjectPtr out = output(a[11], v.out_shape, c.device);
  auto* op = c.plain<uint16_t>(out, at::kHalf, v.out_shape);
  if (!c.good) return not_here();
  return finish(lib.gated(g.values, g.masks, u.values, u.masks, v.x, op, g.rows, g.cols, v.batch, int(N), int(M), gate_bias,
                          up_bias, activation, ws, bytes, c.stream),
                std::move(out));
}

// Rows as block.py's _spaced takes them; fp32: allowed, and whether they are.
struct Spaced {
  void* at = nullptr;
  int64_t tokens = 1, heads = 1, width = 0, stride = 0;
  bool fp32 = false;
  at::IntArrayRef shape;
};
Spaced spaced(Call& c, PyObject* o, bool fp32) {
  Spaced s;
  if (!c.good || !THPVariable_Check(o)) {
    c.good = false;
    return s;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  s.fp32 = t.scalar_type() == at::kFloat;
  const int64_t dims = t.dim();
  if ((s.fp32 ? !fp32 : t.scalar_type() != at::kHalf) || !t.is_cuda() || t.get_device() != c.device || dims < 1 || dims > 4) {
    c.good = false;
    return s;
  }
  const auto size = t.sizes(), step = t.strides();
  s.shape = size;
  s.width = size[dims - 1];
  if (dims > 2) s.heads = size[dims - 2];
  const int64_t row = s.heads * s.width;
  if ((step[dims - 1] != 1 && s.width > 1) || (dims > 2 && step[dims - 2] != s.width && s.heads > 1)) c.good = false;
  s.stride = row;
  if (dims == 2 || dims == 3 || (dims == 4 && size[1] == 1)) {
    s.tokens = size[0];
    if (size[0] > 1) s.stride = step[0];
  } else if (dims == 4) {
    if (size[0] > 1 && step[0] != size[1] * step[1]) c.good = false;
    s.tokens = size[0] * size[1];
    s.stride = step[1];
  }
  s.at = t.data_ptr();
  return s;
}

// (x, weight, bias, kind, offset, eps, out)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  if (n != 7 || c.first(a[0]) == nullptr) return not_here();
  const Spaced x = spaced(c, a[0], true);
  if (!c.good || !same_shape(a[6], THPVariable_Unpack(a[0]))) return not_here();
  auto* weight = c.plain<uint16_t>(a[1], at::kHalf, {x.width}, true);
  auto* bias = c.plain<uint16_t>(a[2], at::kHalf, {x.width}, true);
  const int kind = int(c.whole(a[3]));
  const float offset = float(c.number(a[4])), eps = float(c.number(a[5]));
  if (!c.good) return not_here();
  THPObjectPtr out = output(a[6], x.shape, c.device);
  const Spaced y = spaced(c, out, false);
  if (!c.good) return not_here();
  return finish(lib.norm(x.at, static_cast<uint16_t*>(y.at), weight, bias, x.tokens, x.heads, x.width, x.stride, y.stride,
                         x.fp32, kind, offset, eps, c.stream),
                std::move(out));
}

// (x, branch, weight, bias, post, gate, scale, kind, offset, eps, h, out)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  if (n != 12 || c.first(a[0]) == nullptr || a[1] == Py_None) return not_here();
  const Spaced x = spaced(c, a[0], true);
  if (!c.good) return not_here();
  const at::Tensor& t = THPVariable_Unpack(a[0]);
  if (t.dim() > 2 || !same_shape(a[1], t) || !same_shape(a[10], t) || !same_shape(a[11], t)) return not_here();
  const Spaced branch = spaced(c, a[1], false);
  uint16_t* vec[4];   // weight, bias, post, and a gate for all rows
  for (int i = 0; i < 3; ++i) vec[i] = c.plain<uint16_t>(a[2 + i], at::kHalf, {x.width}, true);
  int64_t gate_stride = 0;
  if (c.good && THPVariable_Check(a[5]) && THPVariable_Unpack(a[5]).dim() == 2) {
    if (!same_shape(a[5], t)) return not_here();
    const Spaced gate = spaced(c, a[5], false);
    vec[3] = static_cast<uint16_t*>(gate.at);
    gate_stride = gate.stride;
  } else {
    vec[3] = c.plain<uint16_t>(a[5], at::kHalf, {x.width}, true);
  }
  const float scale = float(c.number(a[6]));
  const int kind = int(c.whole(a[7]));
  const float offset = float(c.number(a[8])), eps = float(c.number(a[9]));
  if (!c.good) return not_here();
  THPObjectPtr h = a[10] != Py_None ? output(a[10], x.shape, c.device)
                                    : THPObjectPtr(THPVariable_Wrap(made(x.shape, t.scalar_type(), c.device)));
  THPObjectPtr out = output(a[11], x.shape, c.device);
  const Spaced hs = spaced(c, h, x.fp32), ys = spaced(c, out, false);
  if (!c.good || hs.fp32 != x.fp32) return not_here();
  if (lib.block_norm(x.at, static_cast<uint16_t*>(branch.at), hs.at, static_cast<uint16_t*>(ys.at), vec[2], vec[3], vec[0],
                     vec[1], x.tokens, x.width, x.stride, branch.stride, hs.stride, ys.stride, gate_stride, x.fp32, kind,
                     scale, offset, eps, c.stream) != 0)
    return not_here();
  return PyTuple_Pack(2, out.get(), h.get());
}

// (logits, tokens, top, scale, workspace)
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  const at::Tensor* t = n == 5 ? c.first(a[0]) : nullptr;
  if (t == nullptr || t->dim() != 2) return not_here();
  const Spaced x = spaced(c, a[0], true);
  if (!c.good) return not_here();
  auto* tokens = c.plain<int32_t>(a[1], at::kInt, {x.tokens}, true);
  const int64_t top = c.whole(a[2]);
  const float scale = float(c.number(a[3]));
  size_t bytes = 0;
  char* ws = workspace(c, a[4], &bytes);
  if (!c.good || top < 0 || top > NM_MAX_TOP) return not_here();
  at::Tensor logprob, best, best_logprobs;
  const at::Tensor entropy = made({x.tokens}, at::kFloat, c.device);
  if (tokens != nullptr) logprob = made({x.tokens}, at::kFloat, c.device);
  if (top > 0) {
    best = made({x.tokens, top}, at::kInt, c.device);
    best_logprobs = made({x.tokens, top}, at::kFloat, c.device);
  }
  auto at_of = [](const at::Tensor& m) { return m.defined() ? m.data_ptr() : nullptr; };
  if (lib.logprobs(x.at, tokens, static_cast<float*>(at_of(logprob)), static_cast<float*>(at_of(entropy)),
                   static_cast<int32_t*>(at_of(best)), static_cast<float*>(at_of(best_logprobs)), x.tokens, x.width, x.stride,
                   top, !x.fp32, scale, ws, bytes, c.stream) != 0)
    return not_here();
  auto given = [](const at::Tensor& m) { return m.defined() ? THPVariable_Wrap(m) : none().release(); };
  return Py_BuildValue("(NNNN)", given(logprob), given(entropy), given(best), given(best_logprobs));
}

// The functions' addresses in the loaded library, in Library's order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t kCount = sizeof(Library) / sizeof(void*);
  if (n != kCount) {
    PyErr_SetString(PyExc_TypeError, "bind takes one address for each function");
    return nullptr;
  }
  void* at[kCount];
  for (Py_ssize_t i = 0; i < n; ++i) at[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  static_assert(sizeof(at) == sizeof(lib), "");
  std::memcpy(&lib, at, sizeof(lib));
  Py_RETURN_NONE;
}

// No C++ exception (memory that runs out) leaves a function.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception&) {
    PyErr_Clear();
    return not_here();
  }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"),
                         method<rope>("nm_rope"),
                         method<kv_append>("nm_kv_append"),
                         method<rope_kv_append>("nm_rope_kv_append"),
                         method<kv_read>("nm_kv_read"),
                         method<kv_compact>("nm_kv_compact"),
                         method<tree_attention>("nm_tree_attention"),
                         method<verify_chain>("nm_verify_chain"),
                         method<verify_tree>("nm_verify_tree"),
                         method<linear>("nm_linear"),
                         method<gated>("nm_gated"),
                         method<norm>("nm_norm"),
                         method<block_norm>("nm_block_norm"),
                         method<logprobs>("nm_logprobs"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_nmtorch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__nmtorch() { return PyModule_Create(&module); }
