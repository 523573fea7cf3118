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
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
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
  decltype(&sffn_quantize_int4) quantize_int4 = nullptr;
  decltype(&sffn_dequantize_int4) dequantize_int4 = nullptr;
  decltype(&sffn_int4_workspace) int4_workspace = nullptr;
  decltype(&sffn_matmul_int4) matmul_int4 = nullptr;
  decltype(&sffn_gated_up_int4) gated_up_int4 = nullptr;
  decltype(&sffn_gated_up) gated_up = nullptr;
  decltype(&sffn_gated_up_backward_workspace) gated_up_backward_workspace = nullptr;
  decltype(&sffn_gated_up_backward) gated_up_backward = nullptr;
  decltype(&sffn_last_error) last_error = nullptr;
} g;

// A tensor that the call can read as it is: of that type and rank, on that
// device, dense where asked, nothing recorded of it (but for a gradient, where
// the call has one).
bool takes(PyObject* o, at::ScalarType type, int64_t dim, int device, bool dense, const Tensor** out, bool grad = false) {
  if (!THPVariable_Check(o)) return false;
  const Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type || t.dim() != dim || !t.is_cuda() || (!grad && t.requires_grad()) ||
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

// The N addresses that a bind function takes.
template <int N>
bool addresses(PyObject* const* args, Py_ssize_t n, std::array<void*, N>* p) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d addresses are taken", N);
    return false;
  }
  for (int i = 0; i < N; ++i) {
    (*p)[i] = PyLong_AsVoidPtr(args[i]);
    if (!(*p)[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return false;
    }
  }
  return true;
}

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  std::array<void*, 8> p;
  if (!addresses<8>(args, n, &p)) return nullptr;
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

PyObject* bind_block(PyObject*, PyObject* const* args, Py_ssize_t n) {
  std::array<void*, 9> p;
  if (!addresses<9>(args, n, &p)) return nullptr;
  g.quantize_int4 = reinterpret_cast<decltype(g.quantize_int4)>(p[0]);
  g.dequantize_int4 = reinterpret_cast<decltype(g.dequantize_int4)>(p[1]);
  g.int4_workspace = reinterpret_cast<decltype(g.int4_workspace)>(p[2]);
  g.matmul_int4 = reinterpret_cast<decltype(g.matmul_int4)>(p[3]);
  g.gated_up_int4 = reinterpret_cast<decltype(g.gated_up_int4)>(p[4]);
  g.gated_up = reinterpret_cast<decltype(g.gated_up)>(p[5]);
  g.gated_up_backward_workspace = reinterpret_cast<decltype(g.gated_up_backward_workspace)>(p[6]);
  g.gated_up_backward = reinterpret_cast<decltype(g.gated_up_backward)>(p[7]);
  g.last_error = reinterpret_cast<decltype(g.last_error)>(p[8]);
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

// A group of columns that shares a scale: 0 or a multiple of 64 (longer than any row: cut), or -1.
int64_t group_size(PyObject* o) {
  if (!PyLong_CheckExact(o)) return -1;
  const int64_t v = whole(o);
  return v < 0 || v % 64 ? -1 : v < SFFN_MAX_SUM ? v : SFFN_MAX_SUM;
}

// Packed codes [N, K / 2] and their scales [N, G].
bool takes_codes(PyObject* codes, PyObject* scales, int64_t group, int device, const Tensor** q, const Tensor** s) {
  if (!takes(codes, at::kByte, 2, device, true, q)) return false;
  if (!takes(scales, at::kFloat, 2, (*q)->get_device(), true, s)) return false;
  const int64_t N = (*q)->size(0), K = 2 * (*q)->size(1);
  return K > 0 && fits(N) && fits(K) && (*s)->size(0) == N && (*s)->size(1) == (group > 0 ? (K + group - 1) / group : 1);
}

// quantize_int4(w, group) -> (codes, scales)
PyObject* quantize_int4(PyObject* const* args, Py_ssize_t n) {
  const Tensor* w;
  if (n != 2 || !g.quantize_int4 || !takes(args[0], at::kBFloat16, 2, -1, false, &w)) return none();
  const int64_t N = w->size(0), K = w->size(1), group = group_size(args[1]);
  int64_t ld;
  void* stream;
  const int device = device_of(*w, &stream);
  if (device < 0 || group < 0 || !fits(N) || !fits(K) || K < 16 || K % 16 || !pitch(*w, &ld)) return none();
  Tensor q = make({N, K / 2}, at::kByte, device);
  Tensor s = make({N, group > 0 ? (K + group - 1) / group : 1}, at::kFloat, device);
  if (g.quantize_int4(w->data_ptr(), ld, q.data_ptr<uint8_t>(), s.data_ptr<float>(), (int)N, (int)K, (int)group, stream) != SFFN_OK)
    return none();
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(q)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(s)));
  return r;
}

// dequantize_int4(codes, scales, group, f32) -> y
PyObject* dequantize_int4(PyObject* const* args, Py_ssize_t n) {
  const Tensor *q, *s;
  if (n != 4 || !g.dequantize_int4) return none();
  const int64_t group = group_size(args[2]);
  if (group < 0 || !takes_codes(args[0], args[1], group, -1, &q, &s)) return none();
  void* stream;
  const int device = device_of(*q, &stream);
  if (device < 0) return none();
  const int64_t N = q->size(0), K = 2 * q->size(1);
  const bool f32 = args[3] == Py_True;
  Tensor y = make({N, K}, f32 ? at::kFloat : at::kBFloat16, device);
  if (g.dequantize_int4(q->data_ptr<uint8_t>(), s->data_ptr<float>(), y.data_ptr(), K, (int)N, (int)K, (int)group,
                        f32 ? SFFN_F32 : SFFN_BF16, stream) != SFFN_OK)
    return none();
  return THPVariable_Wrap(std::move(y));
}

// matmul_int4(x, wq, sw, group, f32) -> y
PyObject* matmul_int4(PyObject* const* args, Py_ssize_t n) {
  const Tensor *x, *q, *s;
  if (n != 5 || !g.matmul_int4 || !takes(args[0], at::kBFloat16, 2, -1, false, &x)) return none();
  const int64_t group = group_size(args[3]);
  void* stream;
  const int device = device_of(*x, &stream);
  if (device < 0 || group < 0 || !takes_codes(args[1], args[2], group, device, &q, &s)) return none();
  const int64_t T = x->size(0), K = x->size(1), N = q->size(0);
  int64_t ld;
  if (!fits(T) || K != 2 * q->size(1) || !pitch(*x, &ld)) return none();
  const bool f32 = args[4] == Py_True;
  const int type = f32 ? SFFN_F32 : SFFN_BF16;
  Tensor y = make({T, N}, f32 ? at::kFloat : at::kBFloat16, device), scratch;
  const size_t nb = g.int4_workspace((int)T, (int)N, (int)K, type, 0);
  if (nb) scratch = make({(int64_t)nb}, at::kByte, device);
  if (g.matmul_int4(x->data_ptr(), ld, q->data_ptr<uint8_t>(), s->data_ptr<float>(), y.data_ptr(), N, (int)T, (int)N, (int)K,
                    (int)group, type, nb ? scratch.data_ptr() : nullptr, nb, stream) != SFFN_OK)
    return none();
  return THPVariable_Wrap(std::move(y));
}

// gated_up_int4(x, w1q, s1, w3q, s3, group, act) -> h
PyObject* gated_up_int4(PyObject* const* args, Py_ssize_t n) {
  const Tensor *x, *q1, *s1, *q3, *s3;
  if (n != 7 || !g.gated_up_int4 || !takes(args[0], at::kBFloat16, 2, -1, false, &x)) return none();
  const int64_t group = group_size(args[5]);
  void* stream;
  const int device = device_of(*x, &stream);
  if (device < 0 || group < 0 || !takes_codes(args[1], args[2], group, device, &q1, &s1) ||
      !takes_codes(args[3], args[4], group, device, &q3, &s3) || q3->sizes() != q1->sizes())
    return none();
  const int64_t T = x->size(0), D = x->size(1), H = q1->size(0);
  int64_t ld;
  if (!fits(T) || D != 2 * q1->size(1) || !pitch(*x, &ld)) return none();
  Tensor h = make({T, H}, at::kBFloat16, device), scratch;
  const size_t nb = g.int4_workspace((int)T, (int)H, (int)D, SFFN_BF16, 1);
  if (nb) scratch = make({(int64_t)nb}, at::kByte, device);
  if (g.gated_up_int4(x->data_ptr(), ld, q1->data_ptr<uint8_t>(), s1->data_ptr<float>(), q3->data_ptr<uint8_t>(),
                      s3->data_ptr<float>(), h.data_ptr(), H, (int)T, (int)D, (int)H, (int)group, (int)whole(args[6]),
                      nb ? scratch.data_ptr() : nullptr, nb, stream) != SFFN_OK)
    return none();
  return THPVariable_Wrap(std::move(h));
}

// The operands of the gated block, checked; false: not an ordinary call.
struct Gated {
  const Tensor *x, *W1, *W3;
  int64_t T, D, H, ld;
  int device;
  void* stream;
};
bool takes_gated(PyObject* const* args, bool grad, Gated* a) {
  if (!takes(args[0], at::kBFloat16, 2, -1, false, &a->x, grad)) return false;
  a->device = device_of(*a->x, &a->stream);
  if (a->device < 0 || !takes(args[1], at::kBFloat16, 2, a->device, true, &a->W1, grad) ||
      !takes(args[2], at::kBFloat16, 2, a->device, true, &a->W3, grad))
    return false;
  a->T = a->x->size(0), a->D = a->x->size(1), a->H = a->W1->size(0);
  return fits(a->T) && fits(a->D) && fits(a->H) && a->W1->size(1) == a->D && a->W3->sizes() == a->W1->sizes() &&
         pitch(*a->x, &a->ld);
}

// h (with z and u, if they are given) of checked operands; a status code.
int run_gated(const Tensor& x, int64_t ld, const Tensor& W1, const Tensor& W3, const Tensor& h, float* z, float* u, int64_t act,
              void* stream) {
  const int64_t H = W1.size(0);
  return g.gated_up(x.data_ptr(), ld, W1.data_ptr(), W3.data_ptr(), h.data_ptr(), H, z, u, H, (int)x.size(0), (int)x.size(1),
                    (int)H, (int)act, stream);
}

// dx, dW1 and dW3 (undefined where not wanted) of checked operands; a status code.
int run_gated_backward(const Tensor& dh, int64_t lddh, const float* z, const float* u, const Tensor& x, int64_t ld,
                       const Tensor& W1, const Tensor& W3, const Tensor& dx, const Tensor& dW1, const Tensor& dW3, int64_t act,
                       int device, void* stream) {
  const int64_t T = x.size(0), D = x.size(1), H = W1.size(0);
  Tensor scratch;
  const size_t nb = g.gated_up_backward_workspace((int)T, (int)H);
  if (nb) scratch = make({(int64_t)nb}, at::kByte, device);
  auto at_of = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  return g.gated_up_backward(dh.data_ptr(), lddh, z, u, H, x.data_ptr(), ld, W1.data_ptr(), W3.data_ptr(), at_of(dx),
                             at_of(dW1), at_of(dW3), (int)T, (int)D, (int)H, (int)act, at_of(scratch), nb, stream);
}

struct Refused {};  // the library does not take a call: operators.py raises its error

// gated_up with its gradient.  z and u, one buffer of [2, T, H], stay in fp32 for the backward pass.
struct GatedUp : torch::autograd::Function<GatedUp> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& x, const Tensor& W1, const Tensor& W3,
                        int64_t act) {
    void* stream;
    int64_t ld = 0;
    const int device = device_of(x, &stream);
    pitch(x, &ld);
    const int64_t T = x.size(0), H = W1.size(0);
    Tensor h = make({T, H}, at::kBFloat16, device), zu = make({2, T, H}, at::kFloat, device);
    float* z = zu.data_ptr<float>();
    if (run_gated(x, ld, W1, W3, h, z, z + T * H, act, stream) != SFFN_OK) throw Refused();
    ctx->save_for_backward({x, W1, W3, zu});
    ctx->saved_data["act"] = act;
    return h;
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx, torch::autograd::variable_list grads) {
    TORCH_CHECK(c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None,
                "the backward pass of gated_up is not captured: gated_up_backward is");
    const auto saved = ctx->get_saved_variables();
    Tensor x = saved[0], W1 = saved[1], W3 = saved[2], zu = saved[3];
    for (Tensor* t : {&x, &W1, &W3, &zu}) {  // hooks on saved tensors keep their values, but not their layout
      const bool right = t->is_cuda() && t->get_device() == x.get_device() &&
                         t->scalar_type() == (t == &zu ? at::kFloat : at::kBFloat16) && t->dim() == (t == &zu ? 3 : 2);
      TORCH_CHECK(right, "a saved tensor of gated_up came back with another type, rank or device");
      if (t != &x) *t = t->contiguous();
    }
    int64_t ld = 0, lddh = 0;
    if (!pitch(x, &ld)) {
      x = x.contiguous();
      ld = x.size(1);
    }
    const int64_t T = x.size(0), D = x.size(1), H = W1.size(0);
    TORCH_CHECK(W1.size(1) == D && W3.sizes() == W1.sizes() && zu.sizes() == at::IntArrayRef({2, T, H}),
                "a saved tensor of gated_up came back with another shape");
    Tensor dh = grads[0].defined() ? grads[0] : at::zeros({T, H}, x.options());
    if (!pitch(dh, &lddh)) {  // an expanded gradient, say
      dh = dh.contiguous();
      lddh = H;
    }
    void* stream;
    const int device = device_of(x, &stream);
    TORCH_CHECK(device >= 0, "the tensors are not on the current device");
    Tensor out[3];
    bool any = false;
    for (int i = 0; i < 3; ++i)
      if (ctx->needs_input_grad(i)) {
        out[i] = make({i ? H : T, D}, at::kBFloat16, device);
        any = true;
      }
    if (any) {
      const float* z = zu.data_ptr<float>();
      TORCH_CHECK(run_gated_backward(dh, lddh, z, z + T * H, x, ld, W1, W3, out[0], out[1], out[2],
                                     ctx->saved_data["act"].toInt(), device, stream) == SFFN_OK,
                  g.last_error());
    }
    if (at::GradMode::is_enabled()) {  // a graph of the backward pass is recorded: it ends here, with an error
      torch::autograd::variable_list real;
      for (auto& t : out)
        if (t.defined()) real.push_back(t.requires_grad_());
      const auto error = std::make_shared<torch::autograd::DelayedError>("gated_up has no second derivative", real.size());
      real = (*error)(std::move(real));
      for (int i = 0, j = 0; i < 3; ++i)
        if (out[i].defined()) out[i] = real[j++];
    }
    return {out[0], out[1], out[2], Tensor()};
  }
};

// gated_up(x, W1, W3, act) -> h
PyObject* gated_up(PyObject* const* args, Py_ssize_t n) {
  Gated a;
  if (n != 4 || !g.gated_up || !takes_gated(args, true, &a)) return none();
  const int64_t act = whole(args[3]);
  if (at::GradMode::is_enabled() && (a.x->requires_grad() || a.W1->requires_grad() || a.W3->requires_grad())) {
    if (!g.gated_up_backward || c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None ||
        a.D % 8 || a.ld % 8 || a.H < 1 || act < SFFN_ACT_RELU || act > SFFN_ACT_SILU ||
        (((uintptr_t)a.x->data_ptr() | (uintptr_t)a.W1->data_ptr() | (uintptr_t)a.W3->data_ptr()) & 15))
      return none();  // refused, or not recorded: operators.py says why
    try {
      return THPVariable_Wrap(GatedUp::apply(*a.x, *a.W1, *a.W3, act));
    } catch (const Refused&) {
      return none();
    }
  }
  Tensor h = make({a.T, a.H}, at::kBFloat16, a.device);
  if (run_gated(*a.x, a.ld, *a.W1, *a.W3, h, nullptr, nullptr, act, a.stream) != SFFN_OK) return none();
  return THPVariable_Wrap(std::move(h));
}

// gated_up_saved(x, W1, W3, act) -> (h, z, u)
PyObject* gated_up_saved(PyObject* const* args, Py_ssize_t n) {
  Gated a;
  if (n != 4 || !g.gated_up || !takes_gated(args, false, &a)) return none();
  Tensor h = make({a.T, a.H}, at::kBFloat16, a.device), z = make({a.T, a.H}, at::kFloat, a.device),
         u = make({a.T, a.H}, at::kFloat, a.device);
  if (run_gated(*a.x, a.ld, *a.W1, *a.W3, h, z.data_ptr<float>(), u.data_ptr<float>(), whole(args[3]), a.stream) != SFFN_OK)
    return none();
  PyObject* r = PyTuple_New(3);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(h)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(z)));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(u)));
  return r;
}

// gated_up_backward(x, W1, W3, act, dh, z, u, need_x, need_1, need_3) -> (dx, dW1, dW3), None where not wanted
PyObject* gated_up_backward(PyObject* const* args, Py_ssize_t n) {
  Gated a;
  const Tensor *dh, *z, *u;
  if (n != 10 || !g.gated_up_backward || !takes_gated(args, false, &a) || !takes(args[4], at::kBFloat16, 2, a.device, false, &dh) ||
      !takes(args[5], at::kFloat, 2, a.device, true, &z) || !takes(args[6], at::kFloat, 2, a.device, true, &u))
    return none();
  int64_t lddh;
  for (const Tensor* t : {dh, z, u})
    if (t->size(0) != a.T || t->size(1) != a.H) return none();
  if (!pitch(*dh, &lddh)) return none();
  Tensor out[3];
  for (int i = 0; i < 3; ++i)
    if (args[7 + i] == Py_True) out[i] = make({i ? a.H : a.T, a.D}, at::kBFloat16, a.device);
  if (run_gated_backward(*dh, lddh, z->data_ptr<float>(), u->data_ptr<float>(), *a.x, a.ld, *a.W1, *a.W3, out[0], out[1], out[2],
                         whole(args[3]), a.device, a.stream) != SFFN_OK)
    return none();
  PyObject* r = PyTuple_New(3);
  if (!r) return nullptr;
  for (int i = 0; i < 3; ++i)
    PyTuple_SET_ITEM(r, i, out[i].defined() ? THPVariable_Wrap(std::move(out[i])) : none());
  return r;
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
    {"bind_block", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_block)), METH_FASTCALL, nullptr},
    method<route>("route"),
    method<quantize_tokens>("quantize_tokens"),
    method<matmul_int8>("matmul_int8"),
    method<grouped_matmul>("grouped_matmul"),
    method<experts_forward>("experts_forward"),
    method<quantize_int4>("quantize_int4"),
    method<dequantize_int4>("dequantize_int4"),
    method<matmul_int4>("matmul_int4"),
    method<gated_up_int4>("gated_up_int4"),
    method<gated_up>("gated_up"),
    method<gated_up_saved>("gated_up_saved"),
    method<gated_up_backward>("gated_up_backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
