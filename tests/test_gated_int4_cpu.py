"""Refusals of the 4-bit products and of the gated block: every check comes before the device is touched."""
import pytest

import activation_sparse_gated_gb300 as sffn
from activation_sparse_gated_gb300 import build as libbuild

P = 1 << 20  # stand-ins for 16-byte aligned device addresses, far apart
X, W, W3, Y, S, S3, WS, Z, U, DH, D1, D3 = (P * 1000 * i for i in range(1, 13))
ARG, ALIGN, DTYPE = sffn.SFFN_ERR_ARG, sffn.SFFN_ERR_ALIGN, sffn.SFFN_ERR_DTYPE
BIG = sffn.SFFN_MAX_ROWS + 1


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return sffn.load()


def call(lib, name, args, bad):
    args = {**args, **bad}
    rc = getattr(lib, name)(*args.values(), None)
    if rc != sffn.SFFN_OK:
        assert name in sffn.sffn_last_error()
    return rc


QUANT = dict(w=X, ldw=64, codes=W, scales=S, N=4, K=64, group=64)


@pytest.mark.parametrize("bad,code", [
    (dict(N=-1), ARG), (dict(N=BIG), ARG), (dict(K=0), ARG), (dict(K=24, ldw=24), ARG), (dict(K=65552, ldw=65552), ARG),
    (dict(ldw=56), ARG), (dict(ldw=68), ARG), (dict(group=-64), ARG), (dict(group=32), ARG), (dict(group=96), ARG),
    (dict(w=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(w=X + 8), ALIGN), (dict(codes=W + 4), ALIGN),
    (dict(scales=S + 2), ALIGN), (dict(codes=X), ARG), (dict(scales=X + 128), ARG), (dict(scales=W + 16), ARG)])
def test_quantize_int4_refuses(lib, bad, code):
    assert call(lib, "sffn_quantize_int4", QUANT, bad) == code


DEQUANT = dict(codes=W, scales=S, y=Y, ldy=64, N=4, K=64, group=64, y_dtype=sffn.SFFN_BF16)


@pytest.mark.parametrize("bad,code", [
    (dict(N=-1), ARG), (dict(K=20, ldy=24), ARG), (dict(ldy=56), ARG), (dict(ldy=68), ARG), (dict(group=1), ARG),
    (dict(y_dtype=sffn.SFFN_I8), DTYPE), (dict(y=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG),
    (dict(y=Y + 8), ALIGN), (dict(codes=W + 8), ALIGN), (dict(scales=S + 1), ALIGN), (dict(y=W), ARG), (dict(y=S), ARG)])
def test_dequantize_int4_refuses(lib, bad, code):
    assert call(lib, "sffn_dequantize_int4", DEQUANT, bad) == code


PLAIN = dict(x=X, ldx=64, wq=W, sw=S, y=Y, ldy=32, T=4, N=32, K=64, group=64, y_dtype=sffn.SFFN_BF16, ws=None, nws=0)
BLOCK = dict(x=X, ldx=64, w1=W, s1=S, w3=W3, s3=S3, h=Y, ldh=32, T=4, D=64, H=32, group=64, act=0, ws=None, nws=0)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), ARG), (dict(T=BIG), ARG), (dict(N=0), ARG), (dict(N=BIG, ldy=BIG), ARG), (dict(K=0), ARG),
    (dict(K=40, ldx=40), ARG), (dict(K=65552, ldx=65552), ARG), (dict(ldx=56), ARG), (dict(ldx=68), ARG), (dict(ldy=31), ARG),
    (dict(group=-1), ARG), (dict(group=100), ARG), (dict(y_dtype=sffn.SFFN_I8), DTYPE), (dict(x=None), ARG),
    (dict(wq=None), ARG), (dict(sw=None), ARG), (dict(y=None), ARG), (dict(x=X + 2), ALIGN), (dict(wq=W + 8), ALIGN),
    (dict(y=Y + 1), ALIGN), (dict(sw=S + 2), ALIGN), (dict(y=X), ARG), (dict(y=W), ARG), (dict(y=S), ARG),
    (dict(T=4096), ARG), (dict(T=4096, ws=WS, nws=64), ARG), (dict(T=4096, ws=WS + 8, nws=1 << 19), ALIGN),
    (dict(T=4096, ws=Y, nws=1 << 19), ARG), (dict(T=4096, ws=X, nws=1 << 19), ARG), (dict(T=4096, ws=W, nws=1 << 19), ARG)])
def test_matmul_int4_refuses(lib, bad, code):
    assert call(lib, "sffn_matmul_int4", PLAIN, bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), ARG), (dict(H=0), ARG), (dict(D=8, ldx=8), ARG), (dict(ldx=60), ARG), (dict(ldh=16), ARG), (dict(act=3), ARG),
    (dict(act=-1), ARG), (dict(group=65), ARG), (dict(x=None), ARG), (dict(w1=None), ARG), (dict(w3=None), ARG),
    (dict(s1=None), ARG), (dict(s3=None), ARG), (dict(h=None), ARG), (dict(w3=W3 + 8), ALIGN), (dict(s3=S3 + 1), ALIGN),
    (dict(h=Y + 1), ALIGN), (dict(h=W3), ARG), (dict(h=S3), ARG), (dict(T=4096), ARG), (dict(T=4096, ws=W3, nws=1 << 19), ARG)])
def test_gated_up_int4_refuses(lib, bad, code):
    assert call(lib, "sffn_gated_up_int4", BLOCK, bad) == code


GATED = dict(x=X, ldx=64, W1=W, W3=W3, h=Y, ldh=32, z=Z, u=U, ldz=32, T=4, D=64, H=32, act=0)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), ARG), (dict(T=BIG), ARG), (dict(D=0), ARG), (dict(D=60), ARG), (dict(D=65544, ldx=65544), ARG), (dict(H=0), ARG),
    (dict(H=65537, ldh=65537, ldz=65537), ARG), (dict(ldx=56), ARG), (dict(ldx=68), ARG), (dict(ldh=31), ARG), (dict(ldz=31), ARG),
    (dict(act=3), ARG), (dict(z=None), ARG), (dict(u=None), ARG), (dict(x=None), ARG), (dict(W1=None), ARG), (dict(W3=None), ARG),
    (dict(h=None), ARG), (dict(x=X + 8), ALIGN), (dict(W1=W + 2), ALIGN), (dict(W3=W3 + 8), ALIGN), (dict(h=Y + 1), ALIGN),
    (dict(z=Z + 2), ALIGN), (dict(h=X), ARG), (dict(z=W), ARG), (dict(u=W3), ARG), (dict(u=Z), ARG), (dict(h=Z), ARG)])
def test_gated_up_refuses(lib, bad, code):
    assert call(lib, "sffn_gated_up", GATED, bad) == code


BACK = dict(dh=DH, lddh=32, z=Z, u=U, ldz=32, x=X, ldx=64, W1=W, W3=W3, dx=Y, dW1=D1, dW3=D3, T=4, D=64, H=32, act=0, ws=WS,
            nws=1 << 19)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), ARG), (dict(D=60), ARG), (dict(H=0), ARG), (dict(act=3), ARG), (dict(lddh=31), ARG), (dict(ldz=31), ARG),
    (dict(ldx=60), ARG), (dict(dh=None), ARG), (dict(z=None), ARG), (dict(u=None), ARG), (dict(x=None), ARG), (dict(W1=None), ARG),
    (dict(dx=Y + 8), ALIGN), (dict(dW1=D1 + 2), ALIGN), (dict(dW3=D3 + 8), ALIGN), (dict(dh=DH + 1), ALIGN), (dict(z=Z + 1), ALIGN),
    (dict(nws=64), ARG), (dict(ws=None), ARG), (dict(ws=WS + 8), ALIGN), (dict(dx=X), ARG), (dict(dW1=W), ARG), (dict(dW3=W3), ARG),
    (dict(dx=DH), ARG), (dict(dW1=Z), ARG), (dict(dW3=U), ARG), (dict(dW1=D3), ARG), (dict(dx=D1), ARG), (dict(dx=WS), ARG),
    (dict(ws=X), ARG), (dict(ws=DH), ARG), (dict(ws=W3), ARG)])
def test_gated_up_backward_refuses(lib, bad, code):
    assert call(lib, "sffn_gated_up_backward", BACK, bad) == code


def test_empty_calls_touch_nothing(lib):
    assert call(lib, "sffn_quantize_int4", QUANT, dict(w=None, codes=None, scales=None, N=0)) == sffn.SFFN_OK
    assert call(lib, "sffn_dequantize_int4", DEQUANT, dict(y=None, codes=None, scales=None, N=0)) == sffn.SFFN_OK
    assert call(lib, "sffn_matmul_int4", PLAIN, dict(x=None, y=None, T=0)) == sffn.SFFN_OK
    assert call(lib, "sffn_gated_up_int4", BLOCK, dict(x=None, h=None, T=0)) == sffn.SFFN_OK
    assert call(lib, "sffn_gated_up", GATED, dict(x=None, h=None, T=0)) == sffn.SFFN_OK
    assert call(lib, "sffn_gated_up_backward", BACK, dict(dx=None, dW1=None, dW3=None)) == sffn.SFFN_OK


def test_workspaces(lib):
    assert lib.sffn_int4_workspace(0, 32, 64, sffn.SFFN_BF16, 0) == 0
    assert lib.sffn_int4_workspace(1, 7168, 2560, sffn.SFFN_F32, 0) == 0
    one = lib.sffn_int4_workspace(4096, 7168, 2560, sffn.SFFN_BF16, 0)
    assert one >= 2 * 7168 * 2560 and lib.sffn_int4_workspace(4096, 7168, 2560, sffn.SFFN_F32, 0) >= 2 * one
    assert lib.sffn_gated_up_backward_workspace(3, 100) == 3 * 2 * 128 * 2


def test_native_calls_decline():
    torch = pytest.importorskip("torch")
    import importlib.util
    if libbuild.build_torch_calls() is None:
        pytest.skip("no PyTorch with CUDA")
    spec = importlib.util.spec_from_file_location("_torch_calls", libbuild.TORCH_CALLS)
    calls = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(calls)
    x, q, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8), torch.ones(8, 1)
    assert calls.quantize_int4(x, 64) is None and calls.quantize_int4(x, None) is None
    assert calls.dequantize_int4(q, s, 64, False) is None and calls.matmul_int4(x, q, s, 64, False) is None
    assert calls.gated_up_int4(x, q, s, q, s, 64, 0) is None and calls.gated_up(x, x, x, 0) is None
    assert calls.gated_up_saved(x, x, x, 0) is None
    assert calls.gated_up_backward(x, x, x, 0, x, s, s, True, True, True) is None
    with pytest.raises(TypeError):
        calls.bind_block(1)
    with pytest.raises(ValueError):
        calls.bind_block(*[0] * 9)


def test_tensor_wrappers_refuse():
    torch = pytest.importorskip("torch")
    x, q, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8), torch.ones(8, 1)
    w = torch.zeros(8, 64, dtype=torch.bfloat16)
    z = torch.zeros(4, 8)
    for make in (lambda: sffn.quantize_int4(w), lambda: sffn.dequantize_int4(q, s), lambda: sffn.matmul_int4(x, q, s),
                 lambda: sffn.gated_up_int4(x, q, s, q, s), lambda: sffn.gated_up(x, w, w), lambda: sffn.gated_up_saved(x, w, w),
                 lambda: sffn.gated_up_backward(x[:, :8], z, z, x, w, w), lambda: sffn.Int4FFN(w, w, w.T)):
        with pytest.raises(ValueError, match="GPU"):
            make()
    with pytest.raises(ValueError, match="type"):
        sffn.quantize_int4(w.float())
    with pytest.raises(ValueError, match="dimensions"):
        sffn.gated_up(x[0], w, w)
    with pytest.raises(ValueError, match="different layers"):
        sffn.Int4FFN(w, w, w)
    with pytest.raises(ValueError, match="act"):
        sffn.Int4FFN(w, w, w.T, act="gelu")


def test_tensor_wrappers_refuse_sizes_past_32_bits():
    torch = pytest.importorskip("torch")
    far = 2 ** 32 + 4  # 4 in 32 bits
    x, w = (torch.empty(n, 64, dtype=torch.bfloat16, device="meta") for n in (far, 8))
    q, s = torch.empty(far, 32, dtype=torch.uint8, device="meta"), torch.empty(far, 1, device="meta")
    for make in (lambda: sffn.quantize_int4(x), lambda: sffn.dequantize_int4(q, s), lambda: sffn.matmul_int4(x, q[:8], s[:8]),
                 lambda: sffn.gated_up_int4(x, q[:8], s[:8], q[:8], s[:8]), lambda: sffn.gated_up(x, w, w),
                 lambda: sffn.gated_up_saved(x, w, w), lambda: sffn.quantize_tokens(x)):
        with pytest.raises(ValueError, match="2\\^31"):
            make()
