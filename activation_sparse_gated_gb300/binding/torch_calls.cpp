// torch_calls.cpp -- the tensor operators' calls without the interpreter: checks,
// output and scratch allocation and the C call of include/sffn.h in one
// function each (CPython's own API; PyTorch supplies tensors and streams).
//
// A small call is a few microseconds on the GPU, and checking a dozen tensors,
// allocating four and passing twenty arguments from Python takes five to ten
// times that.  Each function here takes the ordinary call: tensors of the right
// kind on the current device, the current stream, fresh outputs.  For anything
// else -- and for every refusal -- it returns None, and operators.py goes
// through its own checks, which name what is wrong.
//
// The C entry points are given by address (bind), so this module serves
// whichever build of the library is loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cstddef>
#include <cstdint>

#include "sffn.h"

namespace {

using at::Tensor;

struct Calls {
  decltype(&sffn_route_workspace) route_workspace = nullptr;
  decltype(&sffn_route) route = nullptr;
  decltype(&sffn_quantize_tokens) quantize_tokens = nullptr;
  decltype(&sffn_grouped_workspace) grouped_workspace = nullptr;
  decltype(&sffn_matmul_int8) matmul_int8 = nullptr;
  decltype(&sffn_grouped_matmul) grouped_matmul = nullptr;
  decltype(&sffn_experts_workspace) experts_workspace = nullptr;
  decltype(&sffn_experts_forward) experts_forward = nullptr;
} g;

// A tensor that the call can read as it is: of that type and rank, on that
// device, dense where asked, nothing recorded of it.
bool takes(PyObject* o, at::ScalarType type, int64_t dim, int device, bool dense, const Tensor** out) {
  if (!THPVariable_Check(o)) return false;
  const Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type || t.dim() != dim || !t.is_cuda() || t.requires_grad() ||
      t._fw_grad(0).defined())
    return false;
  if (device >= 0 && t.get_device() != device) return false;
  if (dense && !t.is_contiguous()) return false;
  *out = &t;
  return true;
}

// Row pitch of a matrix with dense rows; false for other strides.
bool pitch(const Tensor& t, int64_t* ld) {
  const int64_t rows = t.size(0), cols = t.size(1);
  if (cols > 1 && t.stride(1) != 1) return false;
  *ld = rows > 1 ? t.stride(0) : cols;
  return *ld >= cols;
}

bool fits(int64_t v) { return v >= 0 && v <= INT32_MAX; }

Tensor make(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
}

// The tensors' device if it is the current one, else -1; its current stream.
int device_of(const Tensor& t, void** stream) {
  const int device = t.get_device();
  const auto s = c10::cuda::getCurrentCUDAStream();
  if (s.device_index() != device) return -1;
  *stream = s.stream();
  return device;
}

PyObject* none() { Py_RETURN_NONE; }

// A Python int, or -1 where it does not fit.
int64_t whole(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) PyErr_Clear();
  return v;
}

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes eight addresses");
    return nullptr;
  }
  std::array<void*, 8> p;
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  g.route_workspace = reinterpret_cast<decltype(g.route_workspace)>(p[0]);
  g.route = reinterpret_cast<decltype(g.route)>(p[1]);
  g.quantize_tokens = reinterpret_cast<decltype(g.quantize_tokens)>(p[2]);
  g.grouped_workspace = reinterpret_cast<decltype(g.grouped_workspace)>(p[3]);
  g.matmul_int8 = reinterpret_cast<decltype(g.matmul_int8)>(p[4]);
  g.grouped_matmul = reinterpret_cast<decltype(g.grouped_matmul)>(p[5]);
  g.experts_workspace = reinterpret_cast<decltype(g.experts_workspace)>(p[6]);
  g.experts_forward = reinterpret_cast<decltype(g.experts_forward)>(p[7]);
  return none();
}

// route(logits, k, flags) -> (weights, ids, offsets, rows)
PyObject* route(PyObject* const* args, Py_ssize_t n) {
  if (n != 3 || !g.route || !THPVariable_Check(args[0]) || !PyLong_CheckExact(args[1])) return none();
  const auto type = THPVariable_Unpack(args[0]).scalar_type();
  const Tensor* z;
  if ((type != at::kFloat && type != at::kBFloat16) || !takes(args[0], type, 2, -1, false, &z)) return none();
  const int64_t T = z->size(0), E = z->size(1), k = whole(args[1]);
  int64_t ld;
  void* stream;
  const int device = device_of(*z, &stream);
  if (device < 0 || !fits(T) || !fits(E) || k < 1 || k > E || !pitch(*z, &ld) || T * k > SFFN_MAX_ROWS) return none();
  Tensor weights = make({T, k}, at::kFloat, device), ids = make({T, k}, at::kInt, device);
  Tensor offsets = make({E + 1}, at::kInt, device), rows = make({T * k}, at::kInt, device), scratch;
  const size_t nb = g.route_workspace((int)T, (int)E, (int)k);
  if (nb) scratch = make({(int64_t)nb}, at::kByte, device);
  if (g.route(z->data_ptr(), ld, weights.data_ptr<float>(), ids.data_ptr<int>(), offsets.data_ptr<int>(),
              rows.data_ptr<int>(), (int)T, (int)E, (int)k, type == at::kFloat ? SFFN_F32 : SFFN_BF16,
              (int)whole(args[2]), nb ? scratch.data_ptr() : nullptr, nb, stream) != SFFN_OK)
    return none();
  PyObject* r = PyTuple_New(4);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(weights)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(ids)));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(offsets)));
  PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(std::move(rows)));
  return r;
}

// quantize_tokens(x) -> (codes, scales)
PyObject* quantize_tokens(PyObject* const* args, Py_ssize_t n) {
  const Tensor* x;
  if (n != 1 || !g.quantize_tokens || !takes(args[0], at::kBFloat16, 2, -1, false, &x)) return none();
  const int64_t T = x->size(0), K = x->size(1);
  int64_t ld;
  void* stream;
  const int device = device_of(*x, &stream);
  if (device < 0 || !fits(T) || !fits(K) || !pitch(*x, &ld)) return none();
  Tensor q = make({T, K}, at::kChar, device), s = make({T}, at::kFloat, device);
  if (g.quantize_tokens(x->data_ptr(), ld, q.data_ptr<int8_t>(), s.data_ptr<float>(), (int)T, (int)K, stream) != SFFN_OK)
    return none();
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(q)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(s)));
  return r;
}

// matmul_int8(xq, sx, wq, sw, f32) -> y
PyObject* matmul_int8(PyObject* const* args, Py_ssize_t n) {
  const Tensor *x, *sx, *w, *sw;
  if (n != 5 || !g.matmul_int8 || !takes(args[0], at::kChar, 2, -1, false, &x)) return none();
  void* stream;
  const int device = device_of(*x, &stream);
  if (device < 0 || !takes(args[1], at::kFloat, 1, device, true, &sx) || !takes(args[2], at::kChar, 2, device, true, &w) ||
      !takes(args[3], at::kFloat, 1, device, true, &sw))
    return none();
  const int64_t T = x->size(0), K = x->size(1), N = w->size(0);
  int64_t ld;
  if (!fits(T) || !fits(K) || !fits(N) || w->size(1) != K || sx->size(0) != T || sw->size(0) != N || !pitch(*x, &ld))
    return none();
  const bool f32 = args[4] == Py_True;
  Tensor y = make({T, N}, f32 ? at::kFloat : at::kBFloat16, device), scratch;
  const size_t nb = g.grouped_workspace((int)T, (int)T, (int)N, (int)K, 1, SFFN_I8);
  if (nb) scratch = make({(int64_t)nb}, at::kByte, device);
  if (g.matmul_int8(x->data_ptr<int8_t>(), ld, sx->data_ptr<float>(), w->data_ptr<int8_t>(), sw->data_ptr<float>(),
                    y.data_ptr(), N, (int)T, (int)N, (int)K, f32 ? SFFN_F32 : SFFN_BF16,
                    nb ? scratch.data_ptr() : nullptr, nb, stream) != SFFN_OK)
    return none();
  return THPVariable_Wrap(std::move(y));
}

// grouped_matmul(x, w, offsets, sx or None, sw or None, index or None, index_div, transposed, f32) -> y
PyObject* grouped_matmul(PyObject* const* args, Py_ssize_t n) {
  if (n != 9 || !g.grouped_matmul || !THPVariable_Check(args[0]) || !PyLong_CheckExact(args[6])) return none();
  const auto type = THPVariable_Unpack(args[0]).scalar_type();
  const bool i8 = type == at::kChar, kn = args[7] == Py_True, f32 = args[8] == Py_True;
  const Tensor *x, *w, *off, *sx = nullptr, *sw = nullptr, *index = nullptr;
  if ((!i8 && type != at::kBFloat16) || !takes(args[0], type, 2, -1, false, &x)) return none();
  void* stream;
  const int device = device_of(*x, &stream);
  if (device < 0 || !takes(args[1], type, 3, device, true, &w) || !takes(args[2], at::kInt, 1, device, true, &off))
    return none();
  const int64_t XR = x->size(0), K = x->size(1), E = w->size(0), N = w->size(kn ? 2 : 1);
  int64_t R = XR, ld;
  if (!fits(XR) || !fits(K) || !fits(E) || !fits(N) || w->size(kn ? 1 : 2) != K || off->size(0) != E + 1 || !pitch(*x, &ld))
    return none();
  if (i8) {
    if (!takes(args[3], at::kFloat, 1, device, true, &sx) || !takes(args[4], at::kFloat, 2, device, true, &sw) ||
        sx->size(0) != XR || sw->size(0) != E || sw->size(1) != N)
      return none();
  } else if (args[3] != Py_None || args[4] != Py_None) {
    return none();
  }
  if (args[5] != Py_None) {
    if (!takes(args[5], at::kInt, 1, device, true, &index)) return none();
    R = index->size(0);
  }
  const int64_t div = whole(args[6]);
  if (!fits(R) || !fits(div)) return none();
  Tensor y = make({R, N}, f32 ? at::kFloat : at::kBFloat16, device), scratch;
  const size_t nb = i8 ? g.grouped_workspace((int)R, (int)XR, (int)N, (int)K, (int)E, SFFN_I8) : 0;
  if (nb) scratch = make({(int64_t)nb}, at::kByte, device);
  const int type_code = i8 ? (int)SFFN_I8 : (int)SFFN_BF16;
  if (g.grouped_matmul(x->data_ptr(), ld, i8 ? sx->data_ptr<float>() : nullptr, w->data_ptr(),
                       i8 ? sw->data_ptr<float>() : nullptr, off->data_ptr<int>(),
                       index ? index->data_ptr<int>() : nullptr, (int)div, y.data_ptr(), N, (int)R, (int)XR, (int)N,
                       (int)K, (int)E, type_code, f32 ? SFFN_F32 : SFFN_BF16, kn ? SFFN_W_KN : 0,
                       nb ? scratch.data_ptr() : nullptr, nb, stream) != SFFN_OK)
    return none();
  return THPVariable_Wrap(std::move(y));
}

// experts_forward(x, routing, W1, W3, W2t, act) -> y
PyObject* experts_forward(PyObject* const* args, Py_ssize_t n) {
  const Tensor *x, *w, *ids, *off, *rows, *W1, *W3, *W2t;
  if (n != 6 || !g.experts_forward || !PyTuple_Check(args[1]) || PyTuple_GET_SIZE(args[1]) != 4 ||
      !takes(args[0], at::kBFloat16, 2, -1, false, &x))
    return none();
  void* stream;
  const int device = device_of(*x, &stream);
  if (device < 0 || !takes(PyTuple_GET_ITEM(args[1], 0), at::kFloat, 2, device, true, &w) ||
      !takes(PyTuple_GET_ITEM(args[1], 1), at::kInt, 2, device, true, &ids) ||
      !takes(PyTuple_GET_ITEM(args[1], 2), at::kInt, 1, device, true, &off) ||
      !takes(PyTuple_GET_ITEM(args[1], 3), at::kInt, 1, device, true, &rows) ||
      !takes(args[2], at::kBFloat16, 3, device, true, &W1) || !takes(args[3], at::kBFloat16, 3, device, true, &W3) ||
      !takes(args[4], at::kBFloat16, 3, device, true, &W2t))
    return none();
  const int64_t T = x->size(0), D = x->size(1), E = W1->size(0), H = W1->size(1), k = w->size(1);
  int64_t ld;
  if (!fits(T) || !fits(D) || !fits(E) || !fits(H) || !fits(k) || W1->size(2) != D || W3->sizes() != W1->sizes() ||
      W2t->sizes() != W1->sizes() || w->size(0) != T || ids->sizes() != w->sizes() || off->size(0) != E + 1 ||
      rows->size(0) != T * k || !pitch(*x, &ld))
    return none();
  Tensor y = make({T, D}, at::kBFloat16, device), scratch;
  const size_t nb = g.experts_workspace((int)T, (int)k, (int)D, (int)H);
  if (nb) scratch = make({(int64_t)nb}, at::kByte, device);
  if (g.experts_forward(x->data_ptr(), ld, w->data_ptr<float>(), ids->data_ptr<int>(), off->data_ptr<int>(),
                        rows->data_ptr<int>(), W1->data_ptr(), W3->data_ptr(), W2t->data_ptr(), y.data_ptr(), (int)T,
                        (int)E, (int)k, (int)D, (int)H, (int)whole(args[5]), nb ? scratch.data_ptr() : nullptr,
                        nb, stream) != SFFN_OK)
    return none();
  return THPVariable_Wrap(std::move(y));
}

// A C++ exception (an allocation that fails, say) becomes PyTorch's Python one.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(args, n);
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    method<route>("route"),
    method<quantize_tokens>("quantize_tokens"),
    method<matmul_int8>("matmul_int8"),
    method<grouped_matmul>("grouped_matmul"),
    method<experts_forward>("experts_forward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
