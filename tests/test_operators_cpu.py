"""Refusals of the mixture-of-experts and 8-bit operators: every check comes before the device is touched."""
import os
import re

import pytest

import activation_sparse_gated_gb300 as sffn
from activation_sparse_gated_gb300 import build as libbuild

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sffn.h")
P = 1 << 20  # stand-ins for 16-byte aligned device addresses, far apart
X, W, Y, S, O, I, WS = (P * 1000 * i for i in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return sffn.load()


def test_operator_constants_match_header():
    text = open(HEADER).read()
    for name in ("SFFN_I8", "SFFN_ROUTE_SIGMOID", "SFFN_ROUTE_NORMALIZE", "SFFN_W_KN"):
        assert int(re.search(rf"\b{name}\s*=\s*(-?\d+)", text).group(1)) == getattr(sffn, name), name
    for name in ("SFFN_MAX_EXPERTS", "SFFN_MAX_CHOICES", "SFFN_MAX_SUM", "SFFN_MAX_ROWS"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(sffn, name), name


def route(lib, logits=X, ld=64, weights=Y, ids=I, offsets=O, rows=S, T=4, E=64, k=8, dtype=0, flags=2, ws=WS, nws=0):
    return lib.sffn_route(logits, ld, weights, ids, offsets, rows, T, E, k, dtype, flags, ws, nws, None)


@pytest.mark.parametrize("bad,code", [
    (dict(E=0, ld=64), sffn.SFFN_ERR_ARG), (dict(E=1025, ld=1025), sffn.SFFN_ERR_ARG), (dict(k=0), sffn.SFFN_ERR_ARG),
    (dict(k=65), sffn.SFFN_ERR_ARG), (dict(k=33), sffn.SFFN_ERR_ARG), (dict(E=4, k=5), sffn.SFFN_ERR_ARG),
    (dict(T=-1), sffn.SFFN_ERR_ARG), (dict(T=1 << 30), sffn.SFFN_ERR_ARG), (dict(ld=63), sffn.SFFN_ERR_ARG),
    (dict(flags=4), sffn.SFFN_ERR_ARG), (dict(dtype=2), sffn.SFFN_ERR_DTYPE), (dict(logits=None), sffn.SFFN_ERR_ARG),
    (dict(offsets=None), sffn.SFFN_ERR_ARG), (dict(rows=None), sffn.SFFN_ERR_ARG),
    (dict(logits=X + 2), sffn.SFFN_ERR_ALIGN), (dict(ids=I + 1), sffn.SFFN_ERR_ALIGN),
    (dict(T=4096, nws=16), sffn.SFFN_ERR_ARG), (dict(T=4096, ws=None), sffn.SFFN_ERR_ARG),
    (dict(T=4096, ws=WS + 4, nws=1 << 20), sffn.SFFN_ERR_ALIGN)])
def test_route_refuses(lib, bad, code):
    assert route(lib, **bad) == code
    assert "sffn_route" in sffn.sffn_last_error()


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), sffn.SFFN_ERR_ARG), (dict(K=0), sffn.SFFN_ERR_ARG), (dict(ld=63), sffn.SFFN_ERR_ARG),
    (dict(x=None), sffn.SFFN_ERR_ARG), (dict(q=None), sffn.SFFN_ERR_ARG), (dict(x=X + 1), sffn.SFFN_ERR_ALIGN),
    (dict(s=S + 2), sffn.SFFN_ERR_ALIGN)])
def test_quantize_refuses(lib, bad, code):
    a = dict(x=X, ld=64, q=Y, s=S, T=4, K=64)
    a.update(bad)
    assert lib.sffn_quantize_tokens(a["x"], a["ld"], a["q"], a["s"], a["T"], a["K"], None) == code


def grouped(lib, **bad):
    a = dict(x=X, ldx=64, sx=S, w=W, sw=S, offsets=O, index=None, div=1, y=Y, ldy=32, R=8, XR=8, N=32, K=64, E=4,
             dtype=sffn.SFFN_BF16, ydt=sffn.SFFN_BF16, flags=0, ws=None, nws=0)
    a.update(bad)
    return lib.sffn_grouped_matmul(*[a[k] for k in ("x", "ldx", "sx", "w", "sw", "offsets", "index", "div", "y", "ldy",
                                                   "R", "XR", "N", "K", "E", "dtype", "ydt", "flags", "ws", "nws")],
                                   None)


@pytest.mark.parametrize("bad,code", [
    (dict(R=-1), sffn.SFFN_ERR_ARG), (dict(XR=7), sffn.SFFN_ERR_ARG), (dict(N=0), sffn.SFFN_ERR_ARG),
    (dict(K=0), sffn.SFFN_ERR_ARG), (dict(K=60), sffn.SFFN_ERR_ARG), (dict(E=0), sffn.SFFN_ERR_ARG),
    (dict(E=1025), sffn.SFFN_ERR_ARG), (dict(ldx=56), sffn.SFFN_ERR_ARG), (dict(ldx=68), sffn.SFFN_ERR_ARG),
    (dict(ldy=31), sffn.SFFN_ERR_ARG), (dict(K=65544, ldx=65544), sffn.SFFN_ERR_ARG),
    (dict(R=(1 << 28) + 1), sffn.SFFN_ERR_ARG), (dict(N=(1 << 28) + 8), sffn.SFFN_ERR_ARG),
    (dict(index=I, div=0), sffn.SFFN_ERR_ARG), (dict(index=I, XR=0), sffn.SFFN_ERR_ARG),
    (dict(dtype=sffn.SFFN_F32), sffn.SFFN_ERR_DTYPE), (dict(ydt=sffn.SFFN_I8), sffn.SFFN_ERR_DTYPE),
    (dict(flags=2), sffn.SFFN_ERR_ARG), (dict(dtype=sffn.SFFN_I8, flags=sffn.SFFN_W_KN), sffn.SFFN_ERR_DTYPE),
    (dict(dtype=sffn.SFFN_I8, K=72, ldx=80), sffn.SFFN_ERR_ARG), (dict(dtype=sffn.SFFN_I8, sx=None), sffn.SFFN_ERR_ARG),
    (dict(dtype=sffn.SFFN_I8, sw=None), sffn.SFFN_ERR_ARG), (dict(flags=sffn.SFFN_W_KN, N=36, ldy=36), sffn.SFFN_ERR_ARG),
    (dict(x=None), sffn.SFFN_ERR_ARG), (dict(offsets=None), sffn.SFFN_ERR_ARG), (dict(x=X + 8), sffn.SFFN_ERR_ALIGN),
    (dict(w=W + 2), sffn.SFFN_ERR_ALIGN), (dict(y=Y + 1), sffn.SFFN_ERR_ALIGN), (dict(offsets=O + 2), sffn.SFFN_ERR_ALIGN),
    (dict(y=X + 64), sffn.SFFN_ERR_ARG), (dict(y=W), sffn.SFFN_ERR_ARG),
    (dict(dtype=sffn.SFFN_I8, R=8192, XR=8192), sffn.SFFN_ERR_ARG),
    (dict(dtype=sffn.SFFN_I8, R=8192, XR=8192, ws=WS, nws=64), sffn.SFFN_ERR_ARG),
    (dict(dtype=sffn.SFFN_I8, R=8192, XR=8192, ws=WS + 8, nws=1 << 24), sffn.SFFN_ERR_ALIGN),
    (dict(dtype=sffn.SFFN_I8, R=8192, XR=8192, ws=Y, nws=1 << 24), sffn.SFFN_ERR_ARG)])
def test_grouped_matmul_refuses(lib, bad, code):
    assert grouped(lib, **bad) == code
    assert "sffn_grouped_matmul" in sffn.sffn_last_error()


def test_empty_calls_touch_nothing(lib):
    assert grouped(lib, R=0) == sffn.SFFN_OK
    assert lib.sffn_matmul_int8(X, 64, S, W, S, Y, 32, 0, 32, 64, sffn.SFFN_BF16, None, 0, None) == sffn.SFFN_OK
    assert lib.sffn_quantize_tokens(None, 64, None, None, 0, 64, None) == sffn.SFFN_OK
    assert experts(lib, T=0) == sffn.SFFN_OK


def test_matmul_int8_refuses(lib):
    assert lib.sffn_matmul_int8(X, 72, S, W, S, Y, 32, 4, 32, 72, sffn.SFFN_BF16, None, 0, None) == sffn.SFFN_ERR_ARG
    assert lib.sffn_matmul_int8(X, 64, None, W, S, Y, 32, 4, 32, 64, sffn.SFFN_BF16, None, 0, None) == sffn.SFFN_ERR_ARG


def experts(lib, **bad):
    a = dict(x=X, ldx=64, weights=S, ids=I, offsets=O, rows=O, W1=W, W3=W, W2t=W, y=Y, T=4, E=8, k=2, D=64, H=48, act=0,
             ws=WS, nws=1 << 20)
    a.update(bad)
    return lib.sffn_experts_forward(*[a[k] for k in ("x", "ldx", "weights", "ids", "offsets", "rows", "W1", "W3", "W2t",
                                                     "y", "T", "E", "k", "D", "H", "act", "ws", "nws")], None)


@pytest.mark.parametrize("bad,code", [
    (dict(act=3), sffn.SFFN_ERR_ARG), (dict(T=-1), sffn.SFFN_ERR_ARG), (dict(H=0), sffn.SFFN_ERR_ARG),
    (dict(E=0), sffn.SFFN_ERR_ARG), (dict(k=9), sffn.SFFN_ERR_ARG), (dict(k=0), sffn.SFFN_ERR_ARG),
    (dict(D=60), sffn.SFFN_ERR_ARG), (dict(D=0), sffn.SFFN_ERR_ARG), (dict(ldx=60), sffn.SFFN_ERR_ARG),
    (dict(ldx=68), sffn.SFFN_ERR_ARG), (dict(x=None), sffn.SFFN_ERR_ARG), (dict(W2t=None), sffn.SFFN_ERR_ARG),
    (dict(ids=None), sffn.SFFN_ERR_ARG), (dict(W1=W + 8), sffn.SFFN_ERR_ALIGN), (dict(y=Y + 8), sffn.SFFN_ERR_ALIGN),
    (dict(weights=S + 1), sffn.SFFN_ERR_ALIGN), (dict(nws=16), sffn.SFFN_ERR_ARG), (dict(ws=None), sffn.SFFN_ERR_ARG),
    (dict(ws=WS + 8), sffn.SFFN_ERR_ALIGN), (dict(y=X), sffn.SFFN_ERR_ARG), (dict(y=W + 64), sffn.SFFN_ERR_ARG)])
def test_experts_forward_refuses(lib, bad, code):
    assert experts(lib, **bad) == code
    assert "sffn_experts_forward" in sffn.sffn_last_error()


def test_workspace_sizes(lib):
    assert sffn.sffn_route_workspace(1, 64, 8) == 0
    assert sffn.sffn_route_workspace(16384, 256, 8) > 0
    assert sffn.sffn_route_workspace(16384, 2000, 8) == 0
    assert sffn.sffn_grouped_workspace(64, 64, 1024, 512, 4, sffn.SFFN_I8) == 0
    assert sffn.sffn_grouped_workspace(8192, 8192, 1024, 512, 4, sffn.SFFN_BF16) == 0
    assert sffn.sffn_grouped_workspace(8192, 8192, 1024, 512, 4, sffn.SFFN_I8) >= 2 * 512 * (8192 + 4 * 1024)
    assert sffn.sffn_experts_workspace(1, 8, 2560, 1024) >= 4 * 8 * 1024
    assert sffn.sffn_experts_workspace(0, 8, 2560, 1024) == 0
    # sizes pass 32 bits
    assert sffn.sffn_experts_workspace(1 << 20, 8, 4096, 14336) > 1 << 33


def test_native_calls_build_load_and_decline(lib):
    """The one-step calls load against the installed PyTorch, and answer None for what they do not take."""
    torch = pytest.importorskip("torch")
    libbuild.build_torch_calls()
    import importlib.util
    spec = importlib.util.spec_from_file_location("_torch_calls", libbuild.TORCH_CALLS)
    calls = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(calls)
    z = torch.zeros(4, 8)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    assert calls.route(z, 2, 0) is None and calls.route(None, 2, 0) is None and calls.route(z) is None
    assert calls.quantize_tokens(x) is None and calls.quantize_tokens(7) is None
    assert calls.matmul_int8(x, z, x, z, False) is None
    assert calls.grouped_matmul(x, w, off, None, None, None, 1, False, False) is None
    assert calls.experts_forward(x, (z, off, off, off), w, w, w, 0) is None
    with pytest.raises(TypeError):
        calls.bind(1, 2)
    with pytest.raises(ValueError):
        calls.bind(*[0] * 8)


def test_tensor_wrappers_refuse():
    torch = pytest.importorskip("torch")
    z, x = torch.zeros(4, 8), torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)
    for call in (lambda: sffn.route(z, 2), lambda: sffn.quantize_tokens(x), lambda: sffn.matmul_int8(q, s, q, s)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="type"):
        sffn.quantize_tokens(z)
    with pytest.raises(ValueError, match="dimensions"):
        sffn.route(z[0], 2)
    with pytest.raises(AttributeError):
        sffn.no_such_operator


def fake_torch(monkeypatch, root, version, libs):
    """What build.py sees of an installed PyTorch of that version with those libraries."""
    d = root / version / "torch"
    (d / "lib").mkdir(parents=True)
    (d / "__init__.py").write_text("")
    (d / "version.py").write_text(f"from typing import Optional\n__version__ = '{version}'\ncuda = '13.0'\n")
    for name in libs:
        (d / "lib" / name).write_text("")
    import importlib.util
    spec = importlib.util.spec_from_file_location("torch", str(d / "__init__.py"))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else None)


def test_build_without_a_cuda_pytorch(monkeypatch, tmp_path):
    """The C library needs no PyTorch: without one, or with one for CPUs, the calls' module is left out."""
    import importlib.util
    with monkeypatch.context() as m:
        m.setattr(importlib.util, "find_spec", lambda name, *a: None)
        assert libbuild.build_torch_calls(force=True) is None
    fake_torch(monkeypatch, tmp_path, "2.11.0+cpu", ["libtorch_cpu.so"])
    assert libbuild.build_torch_calls(force=True) is None


def test_a_failed_module_leaves_the_library_built(monkeypatch):
    made = []

    def fail(force=False):
        raise RuntimeError("no compiler")

    monkeypatch.setattr(libbuild, "build", lambda **k: made.append("lib"))
    monkeypatch.setattr(libbuild, "build_torch_calls", fail)
    with pytest.raises(RuntimeError):
        libbuild.main([])
    assert made == ["lib"]


def test_module_of_another_pytorch_is_not_loaded(monkeypatch, tmp_path):
    """The module's name holds PyTorch's version and Python's ABI, so after an upgrade of either another one is looked for."""
    torch = pytest.importorskip("torch")
    import sysconfig
    from activation_sparse_gated_gb300 import operators
    assert torch.__version__ in libbuild.TORCH_CALLS and sysconfig.get_config_var("SOABI") in libbuild.TORCH_CALLS
    assert operators._calls is None or operators._calls.__file__ == libbuild.TORCH_CALLS
    for version in ("2.12.0+cu130", "2.11.1"):
        with monkeypatch.context() as m:
            fake_torch(m, tmp_path, version, ["libtorch_cuda.so"])
            assert version in libbuild.torch_calls_path() and libbuild.torch_calls_path() != libbuild.TORCH_CALLS


def test_tensor_wrappers_refuse_forward_mode_tangents():
    torch = pytest.importorskip("torch")
    import torch.autograd.forward_ad as fw
    z, x = torch.zeros(4, 8), torch.zeros(4, 64, dtype=torch.bfloat16)
    with fw.dual_level():
        for call in (lambda: sffn.route(fw.make_dual(z, z), 2), lambda: sffn.quantize_tokens(fw.make_dual(x, x))):
            with pytest.raises(ValueError, match="tangent"):
                call()


@pytest.mark.parametrize("bad", [dict(weights=X), dict(ids=X + 4), dict(rows=X + 4 * 64 * 4 - 4), dict(offsets=X + 8)])
def test_route_refuses_outputs_over_its_logits(lib, bad):
    assert route(lib, **bad) == sffn.SFFN_ERR_ARG
    assert "overlaps" in sffn.sffn_last_error()


@pytest.mark.parametrize("q,s", [(X, S), (X + 2 * 4 * 64 - 1, S), (Y, X + 16)])
def test_quantize_refuses_outputs_over_x(lib, q, s):
    assert lib.sffn_quantize_tokens(X, 64, q, s, 4, 64, None) == sffn.SFFN_ERR_ARG
    assert "overlaps" in sffn.sffn_last_error()


@pytest.mark.parametrize("bad", [dict(y=O), dict(index=Y + 64), dict(dtype=sffn.SFFN_I8, sx=Y), dict(dtype=sffn.SFFN_I8, sw=Y + 4)])
def test_grouped_matmul_refuses_y_over_its_tables(lib, bad):
    assert grouped(lib, **bad) == sffn.SFFN_ERR_ARG
    assert "overlaps" in sffn.sffn_last_error()


@pytest.mark.parametrize("bad", [dict(weights=Y), dict(ids=Y + 4), dict(offsets=Y + 8), dict(rows=Y)])
def test_experts_forward_refuses_y_over_its_routing(lib, bad):
    assert experts(lib, **bad) == sffn.SFFN_ERR_ARG
    assert "overlaps" in sffn.sffn_last_error()


def test_a_pytorch_without_a_readable_version_stops_nothing(monkeypatch, tmp_path):
    with monkeypatch.context() as m:
        fake_torch(m, tmp_path, "2.13.0", ["libtorch_cuda.so"])
        os.remove(tmp_path / "2.13.0" / "torch" / "version.py")
        assert libbuild.torch_calls_path().endswith(".so") and libbuild.torch_calls_path() != libbuild.TORCH_CALLS
