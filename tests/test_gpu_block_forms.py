"""The gated block and the 4-bit products in the forms that the launch rules give to real layers, and their refusals.

The rules go by sizes: one or two units and tiles a block or warp, eight to sixteen warps, sums cut over clusters or not, and the
codes themselves or bf16 copies of them.  Each form has a case here on random data, on both sides of its rule.

Tolerances: a product takes sixteen columns a step, seventeen addends of which each is cut off below 2^-24 of the largest at
worst, so K columns are off by at most (K / 2 + 32) 2^-23 of the sum of magnitudes (the joins of parts among the 32).  What
copies round is in the reference: the copies' values themselves.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import activation_sparse_gated_gb300 as sffn  # noqa: E402
from test_gpu_gated_int4 import (ACTS, BF, DEV, check_h, close, gen, meant, no_device_error, randn, unpack,  # noqa: E402,F401
                                 weights4)

pytestmark = pytest.mark.gpu


def copies(T, N, K, f32, gated=False):
    """Whether a call goes through bf16 copies of its weights: such a call has a workspace."""
    return sffn.load().sffn_int4_workspace(T, N, K, sffn.SFFN_F32 if f32 else sffn.SFFN_BF16, int(gated)) > 0


def taken(codes, scales, group, by_copies, split):
    """The matrix in 64 bits that a call multiplies: codes times scales, or its bf16 copies (split: two parts)."""
    if not by_copies:
        return meant(codes, scales, group)
    q = unpack(codes).float()
    f = q * scales.repeat_interleave(group or q.shape[1], 1)[:, :q.shape[1]]
    high = f.to(BF).float()
    if not split:
        return high.double()
    low = (f - high).to(BF).float()
    return high.double() + torch.where(torch.isfinite(low), low, torch.zeros_like(low)).double()


def off(x, w):
    return (x.shape[1] / 2 + 32) * 2.0 ** -23 * (x.double().abs() @ w.abs().T)


def check_matmul(x, codes, scales, group, dtype, by_copies):
    f32 = dtype == "f32"
    assert copies(x.shape[0], codes.shape[0], x.shape[1], f32) == by_copies
    w = taken(codes, scales, group, by_copies, f32)
    close(sffn.matmul_int4(x, codes, scales, group, dtype=dtype), x.double() @ w.T, off(x, w) * (2 if by_copies and f32 else 1))


@pytest.mark.parametrize("T", [1, 5, 8, 9, 13, 16])
@pytest.mark.parametrize("N,K,group", [(4864, 2560, 64), (4865, 2560, 64), (7175, 1040, 128), (9001, 528, None), (2431, 1104, 64),
                                       (2449, 2064, None)])
def test_rows_of_codes(T, N, K, group):
    g = gen(T + N)
    codes, scales = weights4(g, N, K, group)
    for dtype in ("bf16", "f32"):
        check_matmul(randn(g, T, K), codes, scales, group, dtype, False)


@pytest.mark.parametrize("T,dtype", [(17, "bf16"), (24, "f32"), (25, "bf16"), (32, "f32"), (33, "bf16"), (64, "bf16"), (100, "f32"),
                                     (128, "f32")])
@pytest.mark.parametrize("N,K,group", [(300, 2560, 64), (9472, 1056, 64), (9473, 4096, 128), (14337, 2592, None), (40000, 256, 64)])
def test_tiles_of_codes(T, dtype, N, K, group):
    g = gen(T + N)
    codes, scales = weights4(g, N, K, group)
    check_matmul(randn(g, T, K), codes, scales, group, dtype, False)


@pytest.mark.parametrize("T,dtype", [(33, "f32"), (65, "bf16"), (129, "f32"), (300, "bf16"), (700, "f32")])
@pytest.mark.parametrize("N,K,group", [(40, 80, 64), (515, 2560, 128), (7175, 1040, None)])
def test_copies_of_codes(T, dtype, N, K, group):
    g = gen(T + N)
    codes, scales = weights4(g, N, K, group)
    if not copies(T, N, K, dtype == "f32"):
        assert T == 33 and K % 32 == 0
        return
    check_matmul(randn(g, T, K), codes, scales, group, dtype, True)


@pytest.mark.parametrize("T", [1, 8, 13, 16, 17, 24, 32, 100, 128, 129, 300])
@pytest.mark.parametrize("D,H,group", [(1040, 4865, 64), (2560, 7171, 128), (512, 2433, None)])
def test_gated_block_of_codes(T, D, H, group):
    g = gen(T + H)
    one, three = weights4(g, H, D, group), weights4(g, H, D, group)
    x = randn(g, T, D)
    by_copies = copies(T, H, D, False, True)
    assert by_copies == (T > (128 if D % 32 == 0 else 32))
    w1, w3 = (taken(*w, group, by_copies, True) for w in (one, three))
    for act in ACTS:
        h = sffn.gated_up_int4(x, *one, *three, group=group, act=act)
        check_h(h, x.double() @ w1.T, x.double() @ w3.T, 2 * off(x, w1), 2 * off(x, w3), act)


@pytest.mark.parametrize("T,dtype,by_copies", [(3, "f32", False), (20, "f32", False), (70, "f32", False), (64, "bf16", False),
                                               (65, "bf16", True), (129, "f32", True)])
def test_every_nibble_and_odd_scales(T, dtype, by_copies):
    """-8 among the codes; a scale of 0, a NaN one, a negative one; tokens that hold a NaN or an infinity."""
    g = gen(5)
    codes = torch.randint(0, 256, (70, 96), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.rand(70, 3, generator=g, device=DEV) + 0.1
    scales[3], scales[4, 1], scales[7, 2] = 0.0, -2.5, math.nan
    x = randn(g, T, 192)
    x[1, 5], x[2, 9] = math.nan, math.inf
    f32 = dtype == "f32"
    assert copies(T, 70, 192, f32) == by_copies
    w = taken(codes, scales, 64, by_copies, f32)
    y = sffn.matmul_int4(x, codes, scales, dtype=dtype)
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 7]).all() and not torch.isfinite(y[2]).any()
    rows = torch.tensor([t not in (1, 2) for t in range(T)], device=DEV)
    cols = torch.arange(70, device=DEV) != 7
    close(y[rows][:, cols], x[rows].double() @ w[cols].T, 2 * off(x[rows], w[cols]))
    assert (y[rows][:, 3] == 0).all()


@pytest.mark.parametrize("T", [2, 40, 129])
def test_a_nan_scale_reaches_the_units_that_are_live(T):
    g = gen(9)
    one, three = weights4(g, 64, 128, 64), weights4(g, 64, 128, 64)
    three[1][5] = math.nan
    x = randn(g, T, 128)
    x[0] = -x[-1]
    assert copies(T, 64, 128, False, True) == (T == 129)
    z = x.double() @ taken(*one, 64, T == 129, True).T
    for act in ("relu", "rsp"):
        h = sffn.gated_up_int4(x, *one, *three, act=act)
        dead = z[:, 5] < -1e-3
        assert dead.any() and (h[dead, 5] == 0).all() and torch.isnan(h[z[:, 5] > 1e-3, 5]).all()
        assert not torch.isnan(h[:, :5]).any() and not torch.isnan(h[:, 6:]).any()


@pytest.mark.parametrize("T,dtype,by_copies", [(1, "f32", False), (12, "bf16", False), (40, "f32", False), (65, "bf16", True),
                                               (129, "f32", True)])
def test_weights_past_two_gigabytes(T, dtype, by_copies):
    """Bytes of codes pass 2^31 and elements of copies 2^32: random weights, rows on both sides of each border."""
    N, K = 80000, 65536
    g = gen(T)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.rand(N, 1, generator=g, device=DEV) + 0.5
    x = randn(g, T, K)
    assert copies(T, N, K, dtype == "f32") == by_copies
    y = sffn.matmul_int4(x, codes, scales, None, dtype=dtype)
    some = [n for border in (0, 2 ** 31 // (K // 2), 2 ** 32 // K, 2 ** 32 // (2 * K), N) for n in range(border - 20, border + 20)
            if 0 <= n < N]
    some = torch.tensor(sorted(set(some)), device=DEV)
    w = taken(codes[some], scales[some], None, by_copies, dtype == "f32")
    close(y[:, some], x.double() @ w.T, 2 * off(x, w))


def test_a_long_product():
    g = gen(42)
    codes, scales = weights4(g, 14336, 4096, 64)
    check_matmul(randn(g, 2048, 4096), codes, scales, 64, "bf16", True)


@pytest.mark.parametrize("T,D,H", [(1, 2560, 6080), (1, 2560, 6081), (1, 2560, 7169), (1, 24000, 6081), (1, 24000, 801), (2, 1024, 7169),
                                   (2, 24000, 805), (3, 1024, 8191), (4, 24000, 333), (3, 1024, 8200), (4, 2560, 7169)])
@pytest.mark.parametrize("act", ACTS)
def test_gate_first_tokens(T, D, H, act):
    """One and two units a warp, x in shared memory or not, up to the size where the tensor cores take over."""
    g = gen(T + D + H)
    x, W1, W3 = randn(g, T, D), randn(g, H, D) * D ** -0.5, randn(g, H, D) * D ** -0.5
    W1[5:9] = 0  # neighbours whose gates are exactly 0
    W3[5:9, 3] = math.inf
    h = sffn.gated_up(x, W1, W3, act=act)
    assert (h[:, 5:9] == 0).all()
    W3[5:9, 3] = 0
    z, u = x.double() @ W1.double().T, x.double() @ W3.double().T
    dz, du = ((D / 2 + 32) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T) for w in (W1, W3))
    check_h(h, z, u, dz, du, act)


@pytest.mark.parametrize("T,D,H", [(2, 65544, 4), (2, 64, 65537)])
def test_sizes_past_the_limit_raise_the_same_error_with_and_without_gradients(T, D, H):
    g = gen(1)
    x, W1, W3 = randn(g, T, D), randn(g, H, D), randn(g, H, D)
    for leaf in (None, x, W1, W3):
        args = [t.clone().requires_grad_() if t is leaf else t for t in (x, W1, W3)]
        with pytest.raises(sffn.SffnError, match="at most"):
            sffn.gated_up(*args)
