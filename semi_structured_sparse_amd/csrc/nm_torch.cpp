// The quick way from torch tensors to the calls of nm_decode.h: a Python extension that checks
// the arguments as decode.py does, makes the outputs and calls the library, in 3 to 6 us of the
// host where decode.py alone takes 9 to 16, launch and outputs' allocation included (4 is what
// torch takes to fill an empty tensor; a decoding step makes three such calls a layer). Each
// function returns NotImplemented where anything is not as it should be (a check that fails, a
// tensor on another device than the current one, memory that runs out, a call that the library
// refuses); decode.py then goes its own way, whose checks say what it is. Nothing here touches
// tensor data.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <cmath>
#include <cstring>

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
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_nmtorch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__nmtorch() { return PyModule_Create(&module); }
