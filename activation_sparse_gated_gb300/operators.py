"""The mixture-of-experts and 8-bit operators on torch tensors.

Thin wrappers over the handle-free calls of include/sffn.h: they check shapes,
types and strides, allocate outputs and scratch on the stream the call runs on,
and pass pointers.  ``stream`` is a torch stream (default: the current one);
tensors used on another stream than their own are the caller's to order, as
with any torch operation.  Nothing here is differentiable, and a tensor that
requires a gradient is refused while gradients are recorded, one with a
forward-mode tangent always.

Calls are asynchronous.  A wait inside a kernel that runs out (250 ms, where
microseconds are usual) leaves a call's outputs invalid without an error of its
own: ``sffn_check`` waits for a stream and raises if there was one.

The ordinary call (fresh outputs, the current stream) goes through
``_torch_calls`` (binding/torch_calls.cpp), which checks, allocates and calls the
library in one step and answers None for whatever it does not take; the code
here then does the same and names what is wrong.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from functools import lru_cache

import torch
from torch.autograd import forward_ad

from . import (LIB_PATH, SFFN_ACT_RELU, SFFN_ACT_RSP, SFFN_ACT_SILU, SFFN_BF16, SFFN_F32, SFFN_I8, SFFN_OK,
               SFFN_ROUTE_NORMALIZE, SFFN_ROUTE_SIGMOID, SFFN_W_KN, SffnError, load, sffn_last_error, sffn_strerror)
from .build import TORCH_CALLS

_ACT = {"relu": SFFN_ACT_RELU, "rsp": SFFN_ACT_RSP, "silu": SFFN_ACT_SILU}
_SCORE = {"softmax": 0, "sigmoid": SFFN_ROUTE_SIGMOID}
_OUT = {"bf16": (torch.bfloat16, SFFN_BF16), "f32": (torch.float32, SFFN_F32),
        torch.bfloat16: (torch.bfloat16, SFFN_BF16), torch.float32: (torch.float32, SFFN_F32)}


class Routing(tuple):
    """``route``'s result, the four tensors weights [T, k] fp32, ids [T, k], offsets [E + 1] and rows [T * k] (int32)."""

    weights = property(lambda self: self[0])
    ids = property(lambda self: self[1])
    offsets = property(lambda self: self[2])
    rows = property(lambda self: self[3])


def _load_calls():
    spec = importlib.util.spec_from_file_location(__package__ + "._torch_calls", TORCH_CALLS)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


try:
    _calls = _load_calls()
except ImportError:  # not built for this PyTorch: the same calls, slower
    _calls = None
if _calls is not None and os.path.exists(LIB_PATH):
    _calls.bind(*(ctypes.cast(getattr(load(), name), ctypes.c_void_p).value for name in (
        "sffn_route_workspace", "sffn_route", "sffn_quantize_tokens", "sffn_grouped_workspace", "sffn_matmul_int8",
        "sffn_grouped_matmul", "sffn_experts_workspace", "sffn_experts_forward")))


# no stream object in between, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _raw(device):
    if device.index != _get_device():
        raise ValueError(f"the tensors are on {device}, which is not the current device")
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _done(rc):
    if rc != SFFN_OK:
        raise SffnError(rc, sffn_last_error() or sffn_strerror(rc))


def _has_tangent(t):
    return t.is_floating_point() and forward_ad.unpack_dual(t).tangent is not None


def _operand(name, t, dtypes, dim, device=None):
    if (isinstance(t, torch.Tensor) and t.ndim == dim and t.dtype in dtypes and t.is_cuda
            and (device is None or t.device == device) and not t.requires_grad and not _has_tangent(t)):
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, not {t.dim()}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has type {t.dtype}, not {' or '.join(str(d) for d in dtypes)}")
    if _has_tangent(t):
        raise ValueError(f"{name} has a forward-mode tangent: the operators have none")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient: the operators have none")


# scratch sizes depend on the arguments alone
@lru_cache(maxsize=4096)
def _route_bytes(T, E, k):
    return load().sffn_route_workspace(T, E, k)


@lru_cache(maxsize=4096)
def _grouped_bytes(R, XR, N, K, E):
    return load().sffn_grouped_workspace(R, XR, N, K, E, SFFN_I8)


@lru_cache(maxsize=4096)
def _experts_bytes(T, k, D, H):
    return load().sffn_experts_workspace(T, k, D, H)


def _pitch(name, t):
    """Row pitch of a matrix whose rows are dense (a single row or column: any stride will do)."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return t.stride(0) if rows > 1 else cols


def _dense(name, t):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def route(logits, k: int, score: str = "softmax", normalize: bool = True, stream=None) -> Routing:
    """The k largest of each token's logits [T, E] (fp32 or bf16), their weights and their grouping by expert."""
    if stream is None and _calls is not None and score in _SCORE:
        r = _calls.route(logits, k, _SCORE[score] | (SFFN_ROUTE_NORMALIZE if normalize else 0))
        if r is not None:
            return Routing(r)
    if stream is not None:
        with torch.cuda.stream(stream):
            return route(logits, k, score, normalize)
    _operand("logits", logits, (torch.float32, torch.bfloat16), 2)
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score {score!r} is neither 'softmax' nor 'sigmoid'")
    T, E = logits.shape
    if not 1 <= k <= E:
        raise ValueError(f"k={k} outside 1..{E}")
    device = logits.device
    weights = torch.empty((T, k), dtype=torch.float32, device=device)
    ids = torch.empty((T, k), dtype=torch.int32, device=device)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
    rows = torch.empty(T * k, dtype=torch.int32, device=device)
    ws, nb = _scratch(_route_bytes(T, E, k), device)
    flags = (SFFN_ROUTE_SIGMOID if score == "sigmoid" else 0) | (SFFN_ROUTE_NORMALIZE if normalize else 0)
    _done(load().sffn_route(logits.data_ptr(), _pitch("logits", logits), weights.data_ptr(), ids.data_ptr(),
                            offsets.data_ptr(), rows.data_ptr(), T, E, k,
                            SFFN_F32 if logits.dtype == torch.float32 else SFFN_BF16, flags, nb and ws.data_ptr(), nb,
                            _raw(device)))
    return Routing((weights, ids, offsets, rows))


def quantize_tokens(x, stream=None):
    """(codes int8 [T, K], scales fp32 [T]) of bf16 tokens x [T, K]."""
    if stream is None and _calls is not None:
        r = _calls.quantize_tokens(x)
        if r is not None:
            return r
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantize_tokens(x)
    _operand("x", x, (torch.bfloat16,), 2)
    T, K = x.shape
    q = torch.empty((T, K), dtype=torch.int8, device=x.device)
    s = torch.empty(T, dtype=torch.float32, device=x.device)
    _done(load().sffn_quantize_tokens(x.data_ptr(), _pitch("x", x), q.data_ptr(), s.data_ptr(), T, K, _raw(x.device)))
    return q, s


def _scratch(nb, device):
    return (torch.empty(nb, dtype=torch.uint8, device=device) if nb else None), nb


def _result(out, dtype, shape, device):
    if dtype not in _OUT:
        raise ValueError(f"dtype {dtype!r} is neither bf16 nor f32")
    want, code = _OUT[dtype]
    if out is None:
        return torch.empty(shape, dtype=want, device=device), code, shape[1]
    _operand("out", out, (torch.bfloat16, torch.float32), 2, device)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out has shape {tuple(out.shape)}, not {tuple(shape)}")
    return out, _OUT[out.dtype][1], _pitch("out", out)


def matmul_int8(xq, sx, wq, sw, dtype="bf16", out=None, stream=None):
    """y[t, n] = sx[t] sw[n] sum_k xq[t, k] wq[n, k]; codes xq [T, K], wq [N, K], y of ``dtype`` (or ``out``'s)."""
    if stream is None and out is None and _calls is not None and dtype in _OUT:
        y = _calls.matmul_int8(xq, sx, wq, sw, _OUT[dtype][1] == SFFN_F32)
        if y is not None:
            return y
    if stream is not None:
        with torch.cuda.stream(stream):
            return matmul_int8(xq, sx, wq, sw, dtype, out)
    _operand("xq", xq, (torch.int8,), 2)
    device = xq.device
    _operand("wq", wq, (torch.int8,), 2, device)
    _operand("sx", sx, (torch.float32,), 1, device)
    _operand("sw", sw, (torch.float32,), 1, device)
    T, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError(f"wq has {wq.shape[1]} columns, xq {K}")
    if sx.shape[0] != T or sw.shape[0] != N:
        raise ValueError("one scale per token and per row of wq")
    for name, t in (("wq", wq), ("sx", sx), ("sw", sw)):
        _dense(name, t)
    y, code, ldy = _result(out, dtype, (T, N), device)
    ws, nb = _scratch(_grouped_bytes(T, T, N, K, 1), device)
    _done(load().sffn_matmul_int8(xq.data_ptr(), _pitch("xq", xq), sx.data_ptr(), wq.data_ptr(), sw.data_ptr(),
                                  y.data_ptr(), ldy, T, N, K, code, nb and ws.data_ptr(), nb, _raw(device)))
    return y


def grouped_matmul(x, w, offsets, sx=None, sw=None, index=None, index_div: int = 1, transposed: bool = False,
                   dtype="bf16", out=None, stream=None):
    """Row r of expert e (offsets[e] <= r < offsets[e + 1]) of y is w[e] @ x[r]; with ``index``, w[e] @ x[index[r] //
    index_div].  bf16 x [rows, K] and w [E, N, K] ([E, K, N] with ``transposed``), or int8 codes with their scales sx
    [rows] and sw [E, N].  Rows past offsets[E] are not written."""
    if stream is None and out is None and _calls is not None and dtype in _OUT:
        y = _calls.grouped_matmul(x, w, offsets, sx, sw, index, index_div, bool(transposed),
                                  _OUT[dtype][1] == SFFN_F32)
        if y is not None:
            return y
    if stream is not None:
        with torch.cuda.stream(stream):
            return grouped_matmul(x, w, offsets, sx, sw, index, index_div, transposed, dtype, out)
    _operand("x", x, (torch.bfloat16, torch.int8), 2)
    device, i8 = x.device, x.dtype == torch.int8
    _operand("w", w, (x.dtype,), 3, device)
    _operand("offsets", offsets, (torch.int32,), 1, device)
    XR, K = x.shape
    E, N = w.shape[0], w.shape[2 if transposed else 1]
    if w.shape[1 if transposed else 2] != K:
        raise ValueError(f"w {tuple(w.shape)} does not go with x {tuple(x.shape)}")
    if offsets.shape[0] != E + 1:
        raise ValueError(f"offsets has {offsets.shape[0]} entries, not {E + 1}")
    _dense("w", w)
    _dense("offsets", offsets)
    R = XR
    if index is not None:
        _operand("index", index, (torch.int32,), 1, device)
        _dense("index", index)
        R = index.shape[0]
    if i8:
        if sx is None or sw is None:
            raise ValueError("int8 operands need sx and sw")
        _operand("sx", sx, (torch.float32,), 1, device)
        _operand("sw", sw, (torch.float32,), 2, device)
        if sx.shape[0] != XR or tuple(sw.shape) != (E, N):
            raise ValueError("one scale per row of x and per expert and row of w")
        _dense("sx", sx)
        _dense("sw", sw)
    elif sx is not None or sw is not None:
        raise ValueError("scales go with int8 operands")
    y, code, ldy = _result(out, dtype, (R, N), device)
    ws, nb = _scratch(_grouped_bytes(R, XR, N, K, E) if i8 else 0, device)
    _done(load().sffn_grouped_matmul(
        x.data_ptr(), _pitch("x", x), sx.data_ptr() if i8 else None, w.data_ptr(), sw.data_ptr() if i8 else None,
        offsets.data_ptr(), index.data_ptr() if index is not None else None, index_div, y.data_ptr(), ldy, R, XR, N, K,
        E, SFFN_I8 if i8 else SFFN_BF16, code, SFFN_W_KN if transposed else 0,
        nb and ws.data_ptr(), nb, _raw(device)))
    return y


def experts_forward(x, routing, W1, W3, W2t, act: str = "relu", out=None, stream=None):
    """y[t] = sum_j weights[t, j] W2_e (A(W1_e x_t) * (W3_e x_t)) over the choices e = ids[t, j] of ``route``'s result (or of
    its four tensors); x [T, D], W1, W3 and W2t (W2 transposed) [E, H, D], all bf16."""
    if stream is None and out is None and _calls is not None and act in _ACT:
        y = _calls.experts_forward(x, routing, W1, W3, W2t, _ACT[act])
        if y is not None:
            return y
    if stream is not None:
        with torch.cuda.stream(stream):
            return experts_forward(x, routing, W1, W3, W2t, act, out)
    _operand("x", x, (torch.bfloat16,), 2)
    device = x.device
    if act not in _ACT:
        raise ValueError(f"act {act!r} is none of {', '.join(_ACT)}")
    T, D = x.shape
    shape = W1.shape
    for name, t in (("W1", W1), ("W3", W3), ("W2t", W2t)):
        _operand(name, t, (torch.bfloat16,), 3, device)
        if t.shape != shape or shape[2] != D:
            raise ValueError(f"{name} {tuple(t.shape)} does not go with x {tuple(x.shape)} and W1 {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    E, H = shape[0], shape[1]
    weights, ids, offsets, rows = routing
    _operand("weights", weights, (torch.float32,), 2, device)
    _operand("ids", ids, (torch.int32,), 2, device)
    _operand("offsets", offsets, (torch.int32,), 1, device)
    _operand("rows", rows, (torch.int32,), 1, device)
    for name, t in (("weights", weights), ("ids", ids), ("offsets", offsets), ("rows", rows)):
        _dense(name, t)
    if ids.shape != weights.shape or rows.shape[0] != weights.numel():
        raise ValueError("the routing's tensors are of other tokens or choices")
    k = weights.shape[1]
    if weights.shape[0] != T or offsets.shape[0] != E + 1:
        raise ValueError(f"the routing is of {weights.shape[0]} tokens and {offsets.shape[0] - 1} experts, not {T} and {E}")
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=device)
    else:
        _operand("out", out, (torch.bfloat16,), 2, device)
        if tuple(out.shape) != (T, D):
            raise ValueError(f"out has shape {tuple(out.shape)}, not {(T, D)}")
        _dense("out", out)
    ws, nb = _scratch(_experts_bytes(T, k, D, H), device)
    _done(load().sffn_experts_forward(
        x.data_ptr(), _pitch("x", x), weights.data_ptr(), ids.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
        W1.data_ptr(), W3.data_ptr(), W2t.data_ptr(), out.data_ptr(), T, E, k, D, H, _ACT[act], nb and ws.data_ptr(), nb,
        _raw(device)))
    return out


def _parts(w):
    """w as the sum of bf16 matrices [parts, *w.shape]: 8 of its bits each, so one holds bf16, two fp16 and three fp32."""
    parts, rest = [], w.float()
    for _ in range({torch.bfloat16: 1, torch.float16: 2}.get(w.dtype, 3)):
        parts.append(rest.to(torch.bfloat16))
        rest = rest - parts[-1].float()
    return torch.stack(parts)


class MoEFFN:
    """A mixture of gated experts behind its router, ``y = moe(x)`` for x [T, D] bf16.

    ``Wr`` [E, D] is the router's matrix, W1, W3 [E, H, D] and W2 [E, D, H] the experts' weights.  Wr and W2 are laid out
    once, when the layer is made: W2 as [E, H, D], so that a live unit's column is one contiguous row, and Wr as bf16
    parts whose sum it is, for :func:`grouped_matmul`: the logits are sums in fp32 of all of Wr's bits, whatever
    precision the process allows its matrix products.  ``k`` choices a token, ``score`` and ``normalize`` as in
    :func:`route`.  A token that holds a NaN or an infinity does not come out finite.
    """

    def __init__(self, Wr, W1, W3, W2, k: int, act: str = "relu", score: str = "softmax", normalize: bool = True):
        self.Wr = Wr.float()
        self.W1, self.W3 = W1.contiguous(), W3.contiguous()
        self.W2t = W2.transpose(1, 2).contiguous()
        self.k, self.act, self.score, self.normalize = k, act, score, normalize
        parts = _parts(Wr)
        self._shape = tuple(parts.shape[:2])
        self._parts = parts.reshape(1, -1, Wr.shape[1])  # one group of parts * E rows
        self._all = torch.tensor([0, 2 ** 31 - 1], dtype=torch.int32, device=Wr.device)  # its rows, however many

    def route(self, x):
        z = grouped_matmul(x, self._parts, self._all, dtype="f32")
        if self._shape[0] > 1:
            z = z.view(-1, *self._shape).sum(1)
        # a logit of NaN or -inf closes an expert, and with all of them closed a corrupted token would come out as 0: it
        # counts as 0, so that the token has experts, which keep its NaN
        return route(z.nan_to_num_(0.0, 0.0, 0.0), self.k, self.score, self.normalize)

    def forward(self, x):
        return experts_forward(x, self.route(x), self.W1, self.W3, self.W2t, self.act)

    __call__ = forward
