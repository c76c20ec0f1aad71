// bsq_torch.cpp -- the host side of the Python functions around the linear layers, for calls whose time
// is the host's: it checks the tensors, allocates the outputs, takes the current stream and calls the
// library, as the Python code of the same functions does (a block norm of one token: 15 us there).
//
// Every function returns None where anything about its arguments is not plain -- a wrong type, shape,
// stride or device, or a refusal of the library, which has then enqueued nothing. The Python code
// takes over and says what is wrong. A launch that failed returns its error code instead: launches before
// it may have run (clipping in place scales many tensors in several), so the call must not be repeated. The
// library's functions are called by the addresses given to init(): those of the library that the package has
// loaded.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <exception>
#include <vector>

#include "bsq.h"

namespace {

struct Library {
  decltype(&bsq_block_norm) block_norm;
  decltype(&bsq_block_norm_backward) block_norm_backward;
  decltype(&bsq_block_norm_backward_workspace) block_norm_backward_workspace;
  decltype(&bsq_expert_sort) expert_sort;
  decltype(&bsq_expert_capacity) expert_capacity;
  decltype(&bsq_expert_sort_workspace) expert_sort_workspace;
  decltype(&bsq_expert_gather) expert_gather;
  decltype(&bsq_expert_combine) expert_combine;
  decltype(&bsq_expert_combine_backward) expert_combine_backward;
  decltype(&bsq_grad_norm) grad_norm;
  decltype(&bsq_clip_grad_norm) clip_grad_norm;
  decltype(&bsq_clip_grad_norm_workspace) clip_grad_norm_workspace;
} lib;
constexpr int kFunctions = sizeof(Library) / sizeof(void*);

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat;

// Reads one call's arguments; `ok` turns false at the first that is not plain.
struct Args {
  PyObject* const* at;
  Py_ssize_t count;
  bool ok = true;
  int device = -1;
  int status = kNotCalled;  // of the library's call, BSQ_OK or an error
  static constexpr int kNotCalled = 1;

  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : at(args), count(n), ok(n == want) {}

  // a CUDA tensor on the current device, or nullptr for None
  const at::Tensor* tensor(int i) {
    if (!ok || at[i] == Py_None) return nullptr;
    if (!THPVariable_Check(at[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(at[i]);
    if (!t.is_cuda() || t.layout() != at::kStrided) return fail();
    if (device < 0) {
      device = t.get_device();
      if (device != c10::cuda::current_device()) return fail();
    }
    if (t.get_device() != device) return fail();
    return &t;
  }
  const at::Tensor* needed(int i) {
    const at::Tensor* t = tensor(i);
    if (t == nullptr) ok = false;
    return t;
  }
  // a matrix of bf16 or fp32 with consecutive columns, like `other` where there is one
  const at::Tensor* matrix(int i, const at::Tensor* other = nullptr) {
    const at::Tensor* t = tensor(i);
    if (t == nullptr) return nullptr;
    if ((t->scalar_type() != kBf16 && t->scalar_type() != kF32) || t->dim() != 2) return fail();
    if (t->stride(1) != 1 && t->size(1) != 1) return fail();
    if (other != nullptr && (t->scalar_type() != other->scalar_type() || t->sizes() != other->sizes())) return fail();
    return t;
  }
  const at::Tensor* whole(int i, at::ScalarType type) {
    const at::Tensor* t = tensor(i);
    if (t != nullptr && (t->scalar_type() != type || !t->is_contiguous())) return fail();
    return t;
  }
  // one of a call's parameters of `cols` values, all of one type; a gate may have several rows
  const at::Tensor* param(int i, int64_t cols, at::ScalarType* type, int64_t* groups = nullptr) {
    const at::Tensor* t = tensor(i);
    if (t == nullptr) return nullptr;
    const at::ScalarType s = t->scalar_type();
    if ((s != kBf16 && s != kF32) || (*type != at::ScalarType::Undefined && s != *type) || !t->is_contiguous()) return fail();
    *type = s;
    if (groups != nullptr && t->dim() == 2) {
      *groups = t->size(0);
      if (*groups < 1 || t->size(1) != cols) return fail();
    } else if (t->dim() != 1 || t->size(0) != cols) {
      return fail();
    }
    return t;
  }
  double number(int i) {
    if (!ok) return 0.0;
    const double v = PyFloat_AsDouble(at[i]);
    if (v == -1.0 && PyErr_Occurred()) fail();
    return v;
  }
  int64_t integer(int i) {
    if (!ok) return 0;
    const long long v = PyLong_AsLongLong(at[i]);
    if (v == -1 && PyErr_Occurred()) fail();
    return v;
  }
  const at::Tensor* fail() {
    PyErr_Clear();
    ok = false;
    return nullptr;
  }
  // the library's call, true where it was enqueued
  bool done(int rc) { return (status = rc) == BSQ_OK; }
  at::Tensor make(at::IntArrayRef sizes, at::ScalarType type) const {
    return at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)), std::nullopt);
  }
  bsq_stream_t stream() const {
    return reinterpret_cast<bsq_stream_t>(
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
  }
};

const void* address(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
template <typename T>
T* as(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
int64_t row_stride(const at::Tensor* t) { return t == nullptr ? 0 : t->stride(0); }
PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }
template <typename... T>
PyObject* wrap_all(const T&... tensors) {
  PyObject* r = PyTuple_New(sizeof...(tensors));
  if (r == nullptr) return nullptr;
  Py_ssize_t i = 0;
  ((PyTuple_SET_ITEM(r, i++, wrap(tensors))), ...);
  return r;
}

// No exception of the C++ side passes into Python's C code: before the library's call it counts as "not
// plain", after it as an error of its own.
template <PyObject* (*F)(Args&), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  PyObject* r = nullptr;
  Args a(args, n, N);
  try {
    if (a.ok && lib.block_norm != nullptr) r = F(a);
  } catch (const std::exception& e) {
    if (a.status == BSQ_OK) PyErr_SetString(PyExc_RuntimeError, e.what());
    r = nullptr;
  }
  if (r != nullptr || a.status == BSQ_OK) return r;
  PyErr_Clear();
  if (a.status == BSQ_ERR_LAUNCH) return PyLong_FromLong(a.status);
  Py_RETURN_NONE;
}

// h, x, kind, post_norm, post_weight, post_bias, gate, residual_scale, pre_norm, pre_weight, pre_bias, weight_offset, eps
PyObject* block_norm(Args& a) {
  const at::Tensor* x = a.matrix(1);
  if (x == nullptr) return nullptr;
  const at::Tensor* h = a.matrix(0, x);
  const int64_t rows = x->size(0), cols = x->size(1);
  const bool post = a.integer(3) != 0, pre = a.integer(8) != 0;
  at::ScalarType type = at::ScalarType::Undefined;
  bsq_block_norm_args g{};
  g.kind = static_cast<int32_t>(a.integer(2));
  g.rows = rows, g.cols = cols, g.gate_groups = 1;
  const at::Tensor *pw = a.param(4, cols, &type), *pb = a.param(5, cols, &type),
                   *gate = a.param(6, cols, &type, &g.gate_groups), *w = a.param(9, cols, &type), *b = a.param(10, cols, &type);
  g.residual_scale = static_cast<float>(a.number(7));
  g.weight_offset = static_cast<float>(a.number(11));
  g.eps = static_cast<float>(a.number(12));
  if (!a.ok || (h == nullptr && (post || gate != nullptr)) || (!post && (pw != nullptr || pb != nullptr)) ||
      (!pre && (w != nullptr || b != nullptr)))
    return nullptr;
  g.flags = (x->scalar_type() == kF32 ? BSQ_FLAG_SRC_F32 : 0) | (type == kF32 ? BSQ_FLAG_PARAMS_F32 : 0) |
            (post ? BSQ_FLAG_POST_NORM : 0);
  at::Tensor x_out, y;
  if (h != nullptr || g.residual_scale != 1.0f || !pre) x_out = a.make({rows, cols}, x->scalar_type());
  if (pre) y = a.make({rows, cols}, x->scalar_type());
  const at::Tensor stats = a.make({rows, 4}, kF32);
  g.h = address(h), g.x = x->data_ptr(), g.h_stride = row_stride(h), g.x_stride = row_stride(x);
  g.post_weight = address(pw), g.post_bias = address(pb), g.gate = address(gate);
  g.pre_weight = address(w), g.pre_bias = address(b);
  g.x_out = x_out.defined() ? x_out.data_ptr() : nullptr, g.y = y.defined() ? y.data_ptr() : nullptr;
  g.stats = as<float>(stats);
  return a.done(lib.block_norm(&g, a.stream())) ? wrap_all(x_out, y, stats) : nullptr;
}

// dx_out, dy, x_out, h, stats, kind, post_norm, post_weight, post_bias, gate, residual_scale, pre_weight, pre_bias,
// weight_offset, param_grads
PyObject* block_norm_backward(Args& a) {
  const at::Tensor* dy = a.matrix(1);
  const at::Tensor* dxo = a.matrix(0, dy);
  const at::Tensor* like = dy != nullptr ? dy : dxo;
  if (like == nullptr) return nullptr;
  const at::Tensor *x_out = a.matrix(2, like), *h = a.matrix(3, like), *stats = a.whole(4, kF32);
  const int64_t rows = like->size(0), cols = like->size(1);
  const bool post = a.integer(6) != 0, grads = a.integer(14) != 0;
  at::ScalarType type = at::ScalarType::Undefined;
  bsq_block_norm_grad_args g{};
  g.kind = static_cast<int32_t>(a.integer(5));
  g.rows = rows, g.cols = cols, g.gate_groups = 1;
  const at::Tensor *pw = a.param(7, cols, &type), *pb = a.param(8, cols, &type),
                   *gate = a.param(9, cols, &type, &g.gate_groups), *w = a.param(11, cols, &type), *b = a.param(12, cols, &type);
  g.residual_scale = static_cast<float>(a.number(10));
  g.weight_offset = static_cast<float>(a.number(13));
  if (!a.ok || stats == nullptr || stats->dim() != 2 || stats->size(0) != rows || stats->size(1) != 4 ||
      (dy != nullptr && x_out == nullptr) || (h == nullptr && (post || gate != nullptr)) ||
      (!post && (pw != nullptr || pb != nullptr)))
    return nullptr;
  g.flags = (like->scalar_type() == kF32 ? BSQ_FLAG_SRC_F32 : 0) | (type == kF32 ? BSQ_FLAG_PARAMS_F32 : 0) |
            (post ? BSQ_FLAG_POST_NORM : 0);
  const at::Tensor dx = a.make({rows, cols}, like->scalar_type());
  at::Tensor dh, d[5], ws;
  if (h != nullptr) dh = a.make({rows, cols}, like->scalar_type());
  if (grads) {
    const at::Tensor* wanted[5] = {pw, pb, gate, dy != nullptr ? w : nullptr, dy != nullptr ? b : nullptr};
    bool any = false;
    for (int i = 0; i < 5; ++i)
      if (wanted[i] != nullptr) {
        d[i] = a.make(wanted[i]->sizes(), kF32);
        any = true;
      }
    if (any && rows > 0) {
      g.workspace_bytes = lib.block_norm_backward_workspace(g.flags, rows, cols, g.gate_groups);
      ws = a.make({static_cast<int64_t>(g.workspace_bytes)}, at::kByte);
      g.workspace = ws.data_ptr();
    }
  }
  g.dx_out = address(dxo), g.dy = address(dy), g.x_out = address(x_out), g.h = address(h);
  g.dx_out_stride = row_stride(dxo), g.dy_stride = row_stride(dy), g.x_out_stride = row_stride(x_out);
  g.h_stride = row_stride(h);
  g.stats = static_cast<const float*>(address(stats));
  g.post_weight = address(pw), g.post_bias = address(pb), g.gate = address(gate);
  g.pre_weight = address(w), g.pre_bias = address(b);
  g.dx = dx.data_ptr(), g.dh = dh.defined() ? dh.data_ptr() : nullptr;
  float** to[5] = {&g.dpost_weight, &g.dpost_bias, &g.dgate, &g.dpre_weight, &g.dpre_bias};
  for (int i = 0; i < 5; ++i) *to[i] = d[i].defined() ? as<float>(d[i]) : nullptr;
  return a.done(lib.block_norm_backward(&g, a.stream())) ? wrap_all(dx, dh, d[0], d[1], d[2], d[3], d[4]) : nullptr;
}

// ids, experts, align
PyObject* expert_sort(Args& a) {
  const at::Tensor* ids = a.needed(0);
  const int64_t experts = a.integer(1), align = a.integer(2);
  if (!a.ok || !ids->is_contiguous() || ids->dim() != 2) return nullptr;
  if (ids->scalar_type() != at::kLong && ids->scalar_type() != at::kInt) return nullptr;
  const int64_t tokens = ids->size(0), topk = ids->size(1);
  if (experts < 1 || experts > BSQ_MAX_EXPERTS || align < 1 || topk < 1 || tokens > INT32_MAX / topk) return nullptr;
  const int64_t slots = tokens * topk, capacity = lib.expert_capacity(slots, experts, align);
  if (capacity > INT32_MAX) return nullptr;
  const at::Tensor counts = a.make({experts}, at::kInt), offsets = a.make({experts + 1}, at::kInt),
                   position = a.make({tokens, topk}, at::kInt), slot = a.make({capacity}, at::kInt);
  const size_t bytes = lib.expert_sort_workspace(slots, experts);
  at::Tensor ws;
  if (bytes > 0) ws = a.make({static_cast<int64_t>(bytes)}, at::kByte);
  const int rc = lib.expert_sort(ids->scalar_type() == at::kLong ? BSQ_FLAG_IDS_I64 : 0, ids->data_ptr(), tokens, topk,
                                 experts, align, capacity, as<int32_t>(counts), as<int32_t>(offsets),
                                 as<int32_t>(position), as<int32_t>(slot), ws.defined() ? ws.data_ptr() : nullptr,
                                 bytes, a.stream());
  return a.done(rc) ? wrap_all(counts, offsets, position, slot) : nullptr;
}

int source_flag(const at::Tensor* t) { return t->scalar_type() == kF32 ? BSQ_FLAG_SRC_F32 : 0; }

// x, position, slot
PyObject* expert_gather(Args& a) {
  const at::Tensor *x = a.matrix(0), *position = a.whole(1, at::kInt), *slot = a.whole(2, at::kInt);
  if (!a.ok || x == nullptr || position == nullptr || slot == nullptr || position->dim() != 2 || slot->dim() != 1 ||
      position->size(0) != x->size(0))
    return nullptr;
  const at::Tensor out = a.make({slot->size(0), x->size(1)}, x->scalar_type());
  const int rc = lib.expert_gather(source_flag(x), x->data_ptr(), row_stride(x), as<int32_t>(*position),
                                   as<int32_t>(*slot), x->size(0), position->size(1), x->size(1), slot->size(0),
                                   out.data_ptr(), a.stream());
  return a.done(rc) ? wrap(out) : nullptr;
}

// y, position, weights
PyObject* expert_combine(Args& a) {
  const at::Tensor *y = a.matrix(0), *position = a.whole(1, at::kInt), *weights = a.whole(2, kF32);
  if (!a.ok || y == nullptr || position == nullptr || position->dim() != 2 ||
      (weights != nullptr && weights->sizes() != position->sizes()))
    return nullptr;
  const at::Tensor out = a.make({position->size(0), y->size(1)}, y->scalar_type());
  const int rc = lib.expert_combine(source_flag(y), y->data_ptr(), row_stride(y), as<int32_t>(*position),
                                    static_cast<const float*>(address(weights)), position->size(0), position->size(1),
                                    y->size(1), y->size(0), out.data_ptr(), a.stream());
  return a.done(rc) ? wrap(out) : nullptr;
}

// dout, y, position, slot, weights
PyObject* expert_combine_backward(Args& a) {
  const at::Tensor *dout = a.matrix(0), *y = a.matrix(1), *position = a.whole(2, at::kInt), *slot = a.whole(3, at::kInt),
                   *weights = a.whole(4, kF32);
  if (!a.ok || dout == nullptr || y == nullptr || position == nullptr || slot == nullptr || weights == nullptr) return nullptr;
  if (position->dim() != 2 || weights->sizes() != position->sizes() || slot->dim() != 1 || slot->size(0) != y->size(0) ||
      dout->scalar_type() != y->scalar_type() || dout->size(0) != position->size(0) || dout->size(1) != y->size(1))
    return nullptr;
  const at::Tensor dy = a.make({y->size(0), y->size(1)}, y->scalar_type()), dweights = a.make(position->sizes(), kF32);
  const int rc = lib.expert_combine_backward(
      source_flag(y), dout->data_ptr(), row_stride(dout), y->data_ptr(), row_stride(y), as<int32_t>(*position),
      as<int32_t>(*slot), as<float>(*weights), position->size(0), position->size(1), y->size(1), y->size(0), dy.data_ptr(),
      as<float>(dweights), a.stream());
  return a.done(rc) ? wrap_all(dy, dweights) : nullptr;
}

// list of tensors, list of outputs or None, norm kind, max_norm or None, eps
PyObject* grad_norm(Args& a) {
  PyObject *in = a.at[0], *out = a.at[1];
  if (!PyList_Check(in) || PyList_GET_SIZE(in) == 0 || PyList_GET_SIZE(in) > INT32_MAX) return nullptr;
  if (out != Py_None && (!PyList_Check(out) || PyList_GET_SIZE(out) != PyList_GET_SIZE(in))) return nullptr;
  const Py_ssize_t n = PyList_GET_SIZE(in);
  std::vector<bsq_grad_item> items(static_cast<size_t>(n));
  Args list(nullptr, 0, 0);
  auto plain = [&](PyObject* o) -> const at::Tensor* {
    list.at = &o;
    const at::Tensor* t = list.needed(0);
    if (t == nullptr || !t->is_contiguous() || (t->scalar_type() != kBf16 && t->scalar_type() != kF32)) return nullptr;
    return t;
  };
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor* t = plain(PyList_GET_ITEM(in, i));
    if (t == nullptr) return nullptr;
    bsq_grad_item& it = items[static_cast<size_t>(i)];
    it.src = t->data_ptr(), it.dst = t->data_ptr(), it.elems = t->numel(), it.f32 = t->scalar_type() == kF32;
    if (out != Py_None) {
      const at::ScalarType type = t->scalar_type();
      const at::Tensor* o = plain(PyList_GET_ITEM(out, i));
      if (o == nullptr || o->scalar_type() != type || o->numel() != it.elems) return nullptr;
      it.dst = o->data_ptr();
    }
  }
  const int kind = static_cast<int>(a.integer(2));
  const bool clip = a.at[3] != Py_None;
  const float most = clip ? static_cast<float>(a.number(3)) : 0.0f, eps = static_cast<float>(a.number(4));
  if (!a.ok) return nullptr;
  const size_t bytes = lib.clip_grad_norm_workspace(static_cast<int>(n));
  const at::Tensor norm = list.make({}, kF32), ws = list.make({static_cast<int64_t>(bytes)}, at::kByte);
  const int rc = clip ? lib.clip_grad_norm(static_cast<int>(n), items.data(), kind, most, eps, as<float>(norm),
                                           ws.data_ptr(), bytes, list.stream())
                      : lib.grad_norm(static_cast<int>(n), items.data(), kind, as<float>(norm), ws.data_ptr(), bytes,
                                      list.stream());
  return a.done(rc) ? wrap(norm) : nullptr;
}

// The library's functions, by address, in the order of Library.
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kFunctions) {
    PyErr_SetString(PyExc_TypeError, "init() takes one address for each function");
    return nullptr;
  }
  void* f[kFunctions];
  for (int i = 0; i < kFunctions; ++i) {
    f[i] = PyLong_AsVoidPtr(args[i]);
    if (f[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  std::memcpy(&lib, f, sizeof lib);
  Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction method(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef kMethods[] = {
    {"init", method(init), METH_FASTCALL, nullptr},
    {"block_norm", method(entry<block_norm, 13>), METH_FASTCALL, nullptr},
    {"block_norm_backward", method(entry<block_norm_backward, 15>), METH_FASTCALL, nullptr},
    {"expert_sort", method(entry<expert_sort, 3>), METH_FASTCALL, nullptr},
    {"expert_gather", method(entry<expert_gather, 3>), METH_FASTCALL, nullptr},
    {"expert_combine", method(entry<expert_combine, 3>), METH_FASTCALL, nullptr},
    {"expert_combine_backward", method(entry<expert_combine_backward, 5>), METH_FASTCALL, nullptr},
    {"grad_norm", method(entry<grad_norm, 5>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bsq_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bsq_torch() { return PyModule_Create(&kModule); }
