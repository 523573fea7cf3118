"""4-bit weights and the gated block with its backward pass against plain implementations in 64 bits.

Tolerances count roundings: a result rounded to type t is off by eps(t) / 2 of itself, an fp32 sum of K products by at most
K * 2^-23 of the sum of their magnitudes (each step one rounding, or one truncation on the tensor cores).
"""
import math

import pytest

torch = pytest.importorskip("torch")
import activation_sparse_gated_gb300 as sffn  # noqa: E402

pytestmark = pytest.mark.gpu
BF, DEV = torch.bfloat16, "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ROWS = 32  # most tokens whose products take the codes themselves


@pytest.fixture(autouse=True)
def no_device_error(cuda_ok):
    yield
    sffn.sffn_check()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(BF)


def close(y, ref, bound):
    """|y - ref| <= bound + half a step of y's type, everywhere; NaN and infinities in the same places."""
    y64 = y.double()
    assert y64.shape == ref.shape
    assert torch.equal(torch.isnan(y64), torch.isnan(ref))
    ok = torch.isfinite(ref)
    assert torch.equal(y64[~ok].nan_to_num(), ref[~ok].nan_to_num())
    off = (y64 - ref).abs() - HALF[y.dtype] * 1.01 * ref.abs() - bound
    worst = off[ok].max().item() if ok.any() else 0.0
    assert worst <= 1e-30, f"off by {worst} more than the bound"


# ------------------------------------------------------------------ codes


def plain_codes(w, group):
    """Codes [N, K] and scales [N, G], decided in binary32 on the host."""
    w = w.float().cpu().numpy()
    f32, size = w.dtype.type, group or w.shape[1]
    q, s = [], []
    for k in range(0, w.shape[1], size):
        part = w[:, k:k + size]
        m = abs(part).max(1)
        m[~(m < math.inf)] = math.nan  # (a NaN, or an infinity)
        scale = (m / f32(7))[:, None]
        usable = scale > 0
        q.append(torch.from_numpy((part / scale.clip(min=1e-45)).round().clip(-7, 7) * 1).where(torch.from_numpy(usable), torch.zeros(())))
        s.append(torch.from_numpy(scale))
    return torch.cat(q, 1).to(torch.int8), torch.cat(s, 1)


def unpack(codes):
    n = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1).to(torch.int8)
    return torch.where(n > 7, n - 16, n)


def meant(codes, scales, group):
    q = unpack(codes).double()
    size = group or q.shape[1]
    return q * scales.double().repeat_interleave(size, 1)[:, :q.shape[1]]


def same(a, b):
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(7e30), b.nan_to_num(7e30))


@pytest.mark.parametrize("N,K", [(1, 16), (3, 64), (5, 80), (7, 1008), (16, 1024), (9, 1040), (33, 2560), (2, 16384), (2, 20000),
                                 (1, 65536)])
@pytest.mark.parametrize("group", [64, 128, 192, 256, 512, 1024, 2048, 2112, None, 65536])
def test_codes_and_values(N, K, group):
    w = randn(gen(N + K), N, K)
    w[N // 2, : min(K, 64)] = 0
    w[0, K - 1] = 300.0
    codes, scales = sffn.quantize_int4(w, group)
    q, s = plain_codes(w, group)
    same(scales.cpu(), s)
    assert torch.equal(unpack(codes).cpu(), q)
    v = (q.float() * s.repeat_interleave(group or K, 1)[:, :K])
    same(sffn.dequantize_int4(codes, scales, group, dtype="f32").cpu(), v)
    same(sffn.dequantize_int4(codes, scales, group).cpu().float(), v.to(BF).float())


@pytest.mark.parametrize("group", [64, 512, None])
def test_codes_of_odd_values(group):
    w = randn(gen(3), 12, 1024)
    w[1, 70] = math.nan
    w[2, 900] = math.inf
    w[3, 3] = -math.inf
    w[4] = 0
    w[5] = -0.0
    w[6] = 1e-38 * torch.arange(1024, device=DEV)  # small and subnormal
    w[7] = 2.0 ** -133
    w[8] = 3.3e38
    w[9] = torch.arange(1024, device=DEV) % 15 - 7.0  # whole numbers
    w[10] = (torch.arange(1024, device=DEV) % 29 - 14.0) / 2  # halves: to even
    w[11] = w[10] * 3.0
    codes, scales = sffn.quantize_int4(w, group)
    q, s = plain_codes(w, group)
    same(scales.cpu(), s)
    assert torch.equal(unpack(codes).cpu(), q)


def test_every_bf16_value_beside_every_scale_gets_its_code():
    """All 2^15 magnitudes under 64 group maxima: a code is the correctly rounded quotient's."""
    bits = torch.arange(0x7f80, dtype=torch.int32, device=DEV)
    v = (bits << 16).view(torch.float32).to(BF)
    v = torch.cat((v, torch.zeros(-len(v) % 63, dtype=BF, device=DEV))).view(-1, 63)
    for m in (1e-3, 0.3, 1.0, 7.0, 11.5, 1e4):
        top = torch.full((len(v), 1), m, device=DEV).to(BF)
        w = torch.cat((torch.where(v.abs() <= top, v, torch.zeros_like(v)), top), 1)
        codes, _ = sffn.quantize_int4(w, 64)
        assert torch.equal(unpack(codes).cpu(), plain_codes(w, 64)[0])


def test_every_significand_beside_every_maximum_gets_its_code():
    """The quotient's roundings depend on the two significands and the distance of the exponents: all of them down to 2^-9."""
    v = torch.arange(128, 256, device=DEV).float()
    v = torch.cat([v * 2.0 ** -e for e in range(10)])  # 1280 values below the largest maximum's binade's end
    v = torch.cat((v, torch.zeros(-len(v) % 63, device=DEV))).view(-1, 63)
    rows = []
    for m in range(128, 256):
        top = torch.full((len(v), 1), float(m), device=DEV)
        rows.append(torch.cat((torch.where(v <= m, v, torch.zeros_like(v)), top), 1))
    w = torch.cat(rows) * 2.0 ** -11
    w = torch.cat((w, -w)).to(BF)
    codes, scales = sffn.quantize_int4(w, 64)
    q, s = plain_codes(w, 64)
    same(scales.cpu(), s)
    assert torch.equal(unpack(codes).cpu(), q)


def test_codes_of_strided_rows_and_none():
    w = randn(gen(4), 40, 400)
    a, b = sffn.quantize_int4(w[:, 8:328]), sffn.quantize_int4(w[:, 8:328].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out = torch.full((40, 336), 5.0, dtype=BF, device=DEV)
    sffn.dequantize_int4(*a, out=out[:, :320])
    assert torch.equal(out[:, :320], sffn.dequantize_int4(*a)) and (out[:, 320:] == 5).all()
    codes, scales = sffn.quantize_int4(w[:0])
    assert codes.shape == (0, 200) and scales.shape == (0, 7)
    assert sffn.dequantize_int4(codes, scales).shape == (0, 400)


# ------------------------------------------------------------------ products by 4-bit weights


def weights4(g, N, K, group):
    return sffn.quantize_int4((torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(BF), group)


def bound4(x, w, split, f32):
    """How far a product may be off the exact one before its own rounding; `split`: through bf16 copies."""
    S = x.double().abs() @ w.abs().T
    K = x.shape[1]
    if not split:
        return (K + 16) * 2.0 ** -23 * S
    return (2 * K + 16) * 2.0 ** -23 * S + (2.0 ** -16 if f32 else 2.0 ** -8) * S


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 100, 257])
@pytest.mark.parametrize("N,K,group", [(1, 16, 64), (16, 64, 64), (37, 1008, 128), (100, 2560, 64), (300, 720, None),
                                       (16, 14336, 192), (515, 336, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_matmul_int4(T, N, K, group, dtype):
    g = gen(T * 1000 + N)
    codes, scales = weights4(g, N, K, group)
    x = randn(g, T, K)
    w = meant(codes, scales, group)
    y = sffn.matmul_int4(x, codes, scales, group, dtype=dtype)
    close(y, x.double() @ w.T, bound4(x, w, T > ROWS, dtype == "f32"))


def test_matmul_int4_takes_every_nibble():
    g = gen(5)
    codes = torch.randint(0, 256, (48, 96), generator=g, device=DEV, dtype=torch.uint8)  # -8 among them
    scales = torch.rand(48, 3, generator=g, device=DEV) + 0.1
    w = meant(codes, scales, 64)
    for T in (3, 70):
        x = randn(g, T, 192)
        close(sffn.matmul_int4(x, codes, scales, dtype="f32"), x.double() @ w.T, bound4(x, w, T > ROWS, True))


@pytest.mark.parametrize("T", [4, 20, 60])
def test_matmul_int4_odd_values_stay_in_their_place(T):
    g = gen(6)
    codes, scales = weights4(g, 50, 256, 64)
    scales[3] = 0.0
    scales[7, 2] = math.nan
    x = randn(g, T, 256)
    x[1, 5] = math.nan
    x[2, 9] = math.inf
    w = meant(codes, scales, 64)
    y = sffn.matmul_int4(x, codes, scales, dtype="f32")
    ref = x.double() @ w.T
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 7]).all()
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[1:3] = False
    cols = torch.arange(50, device=DEV) != 7
    close(y[keep][:, cols], ref[keep][:, cols], bound4(x[keep], w[cols], T > ROWS, True))
    assert not torch.isfinite(y[2]).any()  # an infinity meets weights of both signs, or zeros: inf or NaN
    assert (y[keep][:, 3] == 0).all()


@pytest.mark.parametrize("T", [1, 9, 40])
def test_matmul_int4_strided_operands_and_result(T):
    g = gen(7)
    codes, scales = weights4(g, 90, 320, 64)
    big = randn(g, T, 400)
    x = big[:, 40:360]
    y = sffn.matmul_int4(x, codes, scales)
    assert torch.equal(y, sffn.matmul_int4(x.contiguous(), codes, scales))
    out = torch.full((T + 2, 101), 5.0, device=DEV)
    sffn.matmul_int4(x, codes, scales, out=out[:T, :90])
    assert torch.equal(out[:T, :90], sffn.matmul_int4(x, codes, scales, dtype="f32"))
    assert (out[T:] == 5).all() and (out[:, 90:] == 5).all()


def test_int4_no_tokens():
    codes, scales = weights4(gen(8), 64, 128, 64)
    x = torch.empty(0, 128, dtype=BF, device=DEV)
    assert sffn.matmul_int4(x, codes, scales).shape == (0, 64)
    assert sffn.gated_up_int4(x, codes, scales, codes, scales).shape == (0, 64)


def test_int4_codes_past_two_gigabytes():
    """Row offsets of codes pass 31 bits (and elements of the copies 32)."""
    N, K = 80000, 65536  # 2.6 GB of codes
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device=DEV)
    codes[-1] = 0x21  # codes 1 and 2
    scales = torch.full((N, 1), 0.5, device=DEV)
    for T in (2, 33):
        x = torch.ones(T, K, dtype=BF, device=DEV)
        y = sffn.matmul_int4(x, codes, scales, group=None)
        assert (y[:, -1] == K * 1.5 * 0.5).all() and (y[:, :-1] == 0).all()
    last = sffn.dequantize_int4(codes, scales, None)[-1]
    assert (last[0::2] == 0.5).all() and (last[1::2] == 1.0).all()


@pytest.mark.parametrize("T", [3, 12, 40, 300])
def test_int4_products_captured_twice(T):
    """Two graphs of the same calls, each with a workspace of its own, replayed in turn on new tokens."""
    g = gen(10)
    one, three = weights4(g, 300, 512, 64), weights4(g, 300, 512, 64)
    x = randn(g, T, 512)

    def step():
        return sffn.gated_up_int4(x, *one, *three, act="rsp"), sffn.matmul_int4(x, *one), sffn.matmul_int4(x, *three, dtype="f32")

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for seed in (1, 2):
        x.copy_(randn(gen(seed), T, 512))
        want = step()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("T", [1, 3, 8, 11, 27])
def test_int4_the_last_token_is_its_own(T):
    """Idle columns of a tile may hold the last token's values: none of them reach another token."""
    g = gen(11)
    codes, scales = weights4(g, 70, 384, 64)
    x = randn(g, T, 384)
    clean = sffn.matmul_int4(x, codes, scales, dtype="f32")
    x[T - 1] = math.nan
    y = sffn.matmul_int4(x, codes, scales, dtype="f32")
    assert torch.isnan(y[T - 1]).all() and torch.equal(y[:T - 1], clean[:T - 1])


def test_int4_long_sums_and_many_tokens_repeat_their_bits():
    g = gen(12)
    for T, N, K in ((13, 4096, 8192), (100, 515, 2560), (1, 160, 65536), (2, 16, 65520)):
        codes, scales = weights4(g, N, K, 64)
        x = randn(g, T, K)
        y = sffn.matmul_int4(x, codes, scales, dtype="f32")
        w = meant(codes, scales, 64)
        close(y, x.double() @ w.T, bound4(x, w, T > ROWS, True))
        assert all(torch.equal(y, sffn.matmul_int4(x, codes, scales, dtype="f32")) for _ in range(3))


# ------------------------------------------------------------------ the gated block


ACTS = ("relu", "rsp", "silu")


def gate(z, act):
    if act == "relu":
        return torch.where(torch.isnan(z), z, z.clamp(min=0))
    v = torch.where(z == -math.inf, torch.zeros_like(z), z * torch.sigmoid(z))
    return v if act == "silu" else torch.where(z <= 0, torch.zeros_like(v), v)


def slope(z, act):
    if act == "relu":
        return torch.where(torch.isnan(z), z, (z > 0).double())
    p = torch.sigmoid(z)
    v = p + z * p * torch.sigmoid(-z)
    return v if act == "silu" else torch.where(z <= 0, torch.zeros_like(v), v)


def product(z, u, act):
    a = gate(z, act)
    return torch.where(a == 0, torch.zeros_like(a), a * u)


def check_h(h, z, u, dz, du, act):
    """h = A(z) u where z and u are off by dz and du at most; |A'| <= 1.1, the fast exponential 2^-15 of A."""
    a = gate(z, act)
    bound = 1.1 * dz * (u.abs() + du) + a.abs() * du + 2.0 ** -14 * (a.abs() + 1.1 * dz) * (u.abs() + du)
    close(h, product(z, u, act), bound)


@pytest.mark.parametrize("T", [1, 3, 8, 13, 32, 33, 150])
@pytest.mark.parametrize("D,H,group", [(16, 1, 64), (192, 40, 64), (1040, 129, 128), (2560, 300, None)])
@pytest.mark.parametrize("act", ACTS)
def test_gated_up_int4(T, D, H, group, act):
    g = gen(T + D + H)
    one, three = weights4(g, H, D, group), weights4(g, H, D, group)
    x = randn(g, T, D)
    w1, w3 = meant(*one, group), meant(*three, group)
    h = sffn.gated_up_int4(x, *one, *three, group=group, act=act)
    check_h(h, x.double() @ w1.T, x.double() @ w3.T, bound4(x, w1, T > ROWS, True), bound4(x, w3, T > ROWS, True), act)


@pytest.mark.parametrize("T", [2, 40])
def test_gated_up_int4_dead_and_corrupt(T):
    g = gen(9)
    one, three = weights4(g, 64, 128, 64), weights4(g, 64, 128, 64)
    three[1][5] = math.nan  # the up value of unit 5 is NaN
    x = randn(g, T, 128)
    x[0] = -x[-1]  # one of the two keeps the unit, the other does not
    h = sffn.gated_up_int4(x, *one, *three, act="relu")
    z = x.double() @ meant(*one, 64).T
    dead = z[:, 5] < -1e-3
    assert dead.any() and (h[dead, 5] == 0).all() and torch.isnan(h[z[:, 5] > 1e-3, 5]).all()
    x[1] = math.nan
    for act in ACTS:
        assert torch.isnan(sffn.gated_up_int4(x, *one, *three, act=act)[1]).all()


SIZES = [(1, 8, 1), (2, 72, 17), (3, 320, 40), (4, 24000, 9), (5, 64, 100), (16, 384, 129), (77, 384, 1000), (130, 72, 64),
         (300, 264, 330), (1000, 640, 257)]


@pytest.mark.parametrize("T,D,H", SIZES + [(700, 1280, 2000)])
@pytest.mark.parametrize("act", ACTS)
def test_gated_up(T, D, H, act):
    g = gen(T + D + H)
    x, W1, W3 = randn(g, T, D), randn(g, H, D) * D ** -0.5, randn(g, H, D) * D ** -0.5
    z, u = x.double() @ W1.double().T, x.double() @ W3.double().T
    dz, du = ((D + 8) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T) for w in (W1, W3))
    check_h(sffn.gated_up(x, W1, W3, act=act), z, u, dz, du, act)
    h, z32, u32 = sffn.gated_up_saved(x, W1, W3, act=act)
    check_h(h, z, u, dz, du, act)
    close(z32, z, dz)
    close(u32, u, du)


def grads(dh, z, u, x, W1, W3, act):
    """The formula's gradients in 64 bits from z and u, and how far the call's may be off them: dz and du are rounded to
    bf16, A and A' hold to 2^-14 of their terms, the sums are fp32."""
    dh, z, u, x, W1, W3 = (t.double() for t in (dh, z, u, x, W1, W3))
    a, d = gate(z, act), slope(z, act)
    dz, du = dh * u * d, dh * a
    off = 2.0 ** -14 if act != "relu" else 2.0 ** -23
    dzo = 2.0 ** -8 * dz.abs() + 1.3 * off * (dh * u).abs() + 2.0 ** -22 * dz.abs()
    duo = 2.0 ** -8 * du.abs() + off * du.abs() + 2.0 ** -22 * du.abs()
    H, T = z.shape[1], z.shape[0]
    dx = dz @ W1 + du @ W3
    mag = (dz.abs() + dzo) @ W1.abs() + (du.abs() + duo) @ W3.abs()
    out = [(dx, dzo @ W1.abs() + duo @ W3.abs() + (2 * H + 8) * 2.0 ** -23 * mag)]
    for v, o in ((dz, dzo), (du, duo)):
        out.append((v.T @ x, o.T @ x.abs() + (T + 8) * 2.0 ** -23 * ((v.abs() + o).T @ x.abs())))
    return out


@pytest.mark.parametrize("T,D,H", SIZES + [(700, 1280, 2000)])
@pytest.mark.parametrize("act", ACTS)
def test_backward_against_the_formula(T, D, H, act):
    g = gen(T * 3 + D + H)
    x, W1, W3, dh = randn(g, T, D), randn(g, H, D) * D ** -0.5, randn(g, H, D) * D ** -0.5, randn(g, T, H)
    _, z, u = sffn.gated_up_saved(x, W1, W3, act=act)
    got = sffn.gated_up_backward(dh, z, u, x, W1, W3, act=act)
    for y, (ref, bound) in zip(got, grads(dh, z, u, x, W1, W3, act)):
        close(y, ref, bound)


@pytest.mark.parametrize("T,D,H,act", [(4100, 1288, 2601, "rsp"), (4096, 1280, 2600, "silu"), (20000, 136, 5000, "relu")])
def test_training_step_of_pair_tiles(T, D, H, act):
    """Long enough that every product of the step goes to tiles of a pair of blocks; ragged rows, columns and units."""
    g = gen(T + H)
    x, W1, W3, dh = randn(g, T, D), randn(g, H, D) * D ** -0.5, randn(g, H, D) * D ** -0.5, randn(g, T, H)
    h, z, u = sffn.gated_up_saved(x, W1, W3, act=act)
    ref = [x.double() @ w.double().T for w in (W1, W3)]
    off = [(D + 8) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T) for w in (W1, W3)]
    check_h(h, *ref, *off, act)
    close(z, ref[0], off[0])
    close(u, ref[1], off[1])
    got = sffn.gated_up_backward(dh, z, u, x, W1, W3, act=act)
    for y, (want, bound) in zip(got, grads(dh, z, u, x, W1, W3, act)):
        close(y, want, bound)


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(act):
    """The loss sum(dh h) along a direction, by differences in 64 bits, against the gradients' product with it."""
    g = gen(21)
    T, D, H, e = 40, 64, 96, 1e-5
    leaves = [randn(g, T, D), randn(g, H, D) * 0.125, randn(g, H, D) * 0.125]
    dh = randn(g, T, H)
    _, z, u = sffn.gated_up_saved(*leaves, act=act)
    got = sffn.gated_up_backward(dh, z, u, *leaves, act=act)
    bounds = grads(dh, z, u, *leaves, act)

    def loss(x, a, b):
        return (dh.double() * product(x @ a.T, x @ b.T, act)).sum()

    base = [t.double() for t in leaves]
    for i in range(3):
        d = torch.randn(base[i].shape, generator=g, device=DEV, dtype=torch.float64)
        up, down = (loss(*[t + s * e * d if j == i else t for j, t in enumerate(base)]) for s in (1, -1))
        want, have = ((up - down) / (2 * e)).item(), (got[i].double() * d).sum().item()
        room = ((bounds[i][1] + 2.0 ** -8 * bounds[i][0].abs()) * d.abs()).sum().item()
        # a unit whose z crosses 0 within the step, z within e |dz| of it, bends the difference by its slope's jump
        bend = (dh.double() * (base[0] @ base[2].T)).abs() * ((base[0] @ base[1].T).abs() < 1e-3)
        assert abs(want - have) <= room + bend.sum().item() * 10 + 1e-6 * abs(want)


@pytest.mark.parametrize("act", ACTS)
def test_autograd_is_the_backward_call(act):
    g = gen(22)
    x, W1, W3, dh = randn(g, 50, 128), randn(g, 72, 128), randn(g, 72, 128), randn(g, 50, 72)
    _, z, u = sffn.gated_up_saved(x, W1, W3, act=act)
    want = sffn.gated_up_backward(dh, z, u, x, W1, W3, act=act)
    leaves = [t.clone().requires_grad_() for t in (x, W1, W3)]
    h = sffn.gated_up(*leaves, act=act)
    assert torch.equal(h.detach(), sffn.gated_up_saved(x, W1, W3, act=act)[0])
    h.backward(dh)
    for t, w in zip(leaves, want):
        assert torch.equal(t.grad, w)
    for i in range(3):  # one leaf at a time: the others' gradients are not computed
        some = [t.clone().requires_grad_(j == i) for j, t in enumerate((x, W1, W3))]
        sffn.gated_up(*some, act=act).backward(dh)
        assert torch.equal(some[i].grad, want[i]) and all(t.grad is None for j, t in enumerate(some) if j != i)
    both = sffn.gated_up_backward(dh, z, u, x, W1, W3, act=act, need=(False, False, True))
    assert both[0] is None and both[1] is None and torch.equal(both[2], want[2])


def test_autograd_of_a_used_twice_leaf_and_a_view():
    g = gen(23)
    x = randn(g, 30, 64).requires_grad_()
    W = randn(g, 2, 48, 64).requires_grad_()
    h = sffn.gated_up(x, W[0], W[1], act="silu")
    h.sum().backward()  # the gradient of h is one expanded number
    one = torch.ones(30, 48, dtype=BF, device=DEV)
    _, z, u = sffn.gated_up_saved(x.detach(), W.detach()[0], W.detach()[1], act="silu")
    dx, dW1, dW3 = sffn.gated_up_backward(one, z, u, x.detach(), W.detach()[0], W.detach()[1], act="silu")
    assert torch.equal(x.grad, dx) and torch.equal(W.grad, torch.stack((dW1, dW3)))
    V = W.detach()[0].clone().requires_grad_()
    sffn.gated_up(x.detach(), V, V, act="silu").backward(one)  # the same matrix twice: its gradients add up
    _, z, u = sffn.gated_up_saved(x.detach(), V.detach(), V.detach(), act="silu")
    _, a, b = sffn.gated_up_backward(one, z, u, x.detach(), V.detach(), V.detach(), act="silu")
    assert torch.equal(V.grad, a + b)


def test_int4_groups_that_no_scale_has_are_refused():
    x, w = randn(gen(41), 4, 128), randn(gen(42), 8, 128)
    q, s = sffn.quantize_int4(w, None)
    for group in (0, False, -64, 32, 96, 64.0, "64"):
        for call in (lambda: sffn.quantize_int4(w, group), lambda: sffn.dequantize_int4(q, s, group),
                     lambda: sffn.matmul_int4(x, q, s, group), lambda: sffn.gated_up_int4(x, q, s, q, s, group)):
            with pytest.raises(ValueError, match="group"):
                call()


def test_autograd_through_hooks_on_saved_tensors():
    g = gen(43)
    x, W1, W3 = (randn(g, *s).requires_grad_() for s in ((30, 64), (48, 64), (48, 64)))
    dh = randn(g, 30, 48)
    sffn.gated_up(x, W1, W3, act="silu").backward(dh)
    ref = [t.grad.clone() for t in (x, W1, W3)]
    ways = {
        "moved": (lambda t: t.cpu(), lambda t: t.to(DEV)),
        "transposed": (lambda t: t.transpose(-1, -2).contiguous(), lambda t: t.transpose(-1, -2)),
        "spread": (lambda t: t.repeat_interleave(2, -1), lambda t: t[..., ::2])}
    for pack, back in ways.values():
        for t in (x, W1, W3):
            t.grad = None
        with torch.autograd.graph.saved_tensors_hooks(pack, back):
            h = sffn.gated_up(x, W1, W3, act="silu")
        h.backward(dh)
        for t, r in zip((x, W1, W3), ref):
            assert torch.equal(t.grad, r)
    for back in (lambda t: t.cpu(), lambda t: t.double(), lambda t: t[..., :40].contiguous(), lambda t: t[:1]):
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, back):
            h = sffn.gated_up(x, W1, W3, act="silu")
        with pytest.raises(RuntimeError, match="saved tensor|shape|device"):
            h.backward(dh)


def test_gated_up_refuses_what_it_cannot_record():
    g = gen(24)
    x, W1, W3 = randn(g, 4, 64).requires_grad_(), randn(g, 8, 64), randn(g, 8, 64)
    with pytest.raises(ValueError, match="out"):
        sffn.gated_up(x, W1, W3, out=torch.empty(4, 8, dtype=BF, device=DEV))
    with pytest.raises(ValueError, match="gradient"):
        sffn.gated_up_saved(x, W1, W3)
    h = sffn.gated_up(x, W1, W3, act="silu")
    (dx,) = torch.autograd.grad(h.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):  # no second derivative
        dx.float().sum().backward()
    with torch.no_grad():
        assert not sffn.gated_up(x, W1, W3).requires_grad
        sffn.gated_up_saved(x, W1, W3)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x.detach(), torch.ones_like(x))
        with pytest.raises(ValueError, match="tangent"):
            sffn.gated_up(dual, W1, W3)


def test_gated_up_refuses_rows_on_top_of_one_another():
    g = gen(37)
    W1, W3 = randn(g, 8, 64).requires_grad_(), randn(g, 8, 64)
    x = randn(g, 1, 64).expand(4, 64)
    with pytest.raises(sffn.SffnError, match="pitch"):
        sffn.gated_up(x, W1, W3)
    with pytest.raises(sffn.SffnError, match="pitch"):
        sffn.gated_up(x, W1.detach(), W3)
    x = x.contiguous()
    _, z, u = sffn.gated_up_saved(x, W1.detach(), W3)
    with pytest.raises(sffn.SffnError, match="pitch"):
        sffn.gated_up_backward(randn(g, 1, 8).expand(4, 8), z, u, x, W1.detach(), W3)


def test_a_differentiable_call_is_not_captured():
    g = gen(25)
    x, W1, W3 = randn(g, 4, 64).requires_grad_(), randn(g, 8, 64), randn(g, 8, 64)
    sffn.gated_up(x, W1, W3).sum().backward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            sffn.gated_up(x, W1, W3)


@pytest.mark.parametrize("T", [1, 60, 700])
def test_a_captured_training_step_is_replayed(T):
    """Two graphs of the explicit pair, replayed on new inputs while an eager graph of the same leaves lives."""
    g = gen(26)
    D, H = 256, 320
    x, W1, W3, dh = randn(g, T, D), randn(g, H, D), randn(g, H, D), randn(g, T, H)
    leaf = W1.clone().requires_grad_()
    alive = sffn.gated_up(x.clone(), leaf, W3, act="rsp")

    def step():
        h, z, u = sffn.gated_up_saved(x, W1, W3, act="rsp")
        return (h, *sffn.gated_up_backward(dh, z, u, x, W1, W3, act="rsp"))

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for seed in (1, 2):
        x.copy_(randn(gen(seed), T, D))
        dh.copy_(randn(gen(seed + 9), T, H))
        want = step()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    alive.sum().backward()
    assert leaf.grad is not None


def test_backward_zero_and_odd_gradients():
    g = gen(27)
    T, D, H = 40, 64, 48
    x, W1, W3 = randn(g, T, D), randn(g, H, D), randn(g, H, D)
    dh = randn(g, T, H)
    for act in ACTS:
        _, z, u = sffn.gated_up_saved(x, W1, W3, act=act)
        z[0], z[1], z[2] = 0.0, 200.0, -200.0
        z[3], z[4] = math.inf, -math.inf
        u[5, 7] = math.inf
        z[5, 7] = -1.0 if act != "silu" else -200.0  # closed: passes nothing of the infinity
        dz = slope(z.double().clamp(-1e4, 1e4), act) * (dh * u.nan_to_num(0.0, 0.0)).double()
        got = sffn.gated_up_backward(dh, z, u, x, W1, W3, act=act)
        dx3 = got[0][3]
        keep = torch.ones(T, dtype=torch.bool, device=DEV)
        keep[3] = False  # A(inf) = inf: du and this token's dx are no numbers
        assert not torch.isfinite(dx3).all()
        ref, bound = grads(dh[keep], z[keep].clamp(-1e4, 1e4), u[keep].nan_to_num(0.0, 0.0, 0.0), x[keep], W1, W3, act)[0]
        close(got[0][keep], ref, bound)
        assert torch.isfinite(got[1]).all() and dz.isfinite().all()
        if act != "silu":
            assert (got[0][2] == 0).all() and (got[0][4] == 0).all() and (got[0][0] == 0).all()


def test_backward_of_corrupt_tokens_stays_with_them():
    g = gen(28)
    T, D, H = 200, 64, 48
    x, W1, W3, dh = randn(g, T, D), randn(g, H, D), randn(g, H, D), randn(g, T, H)
    _, z, u = sffn.gated_up_saved(x, W1, W3, act="silu")
    clean = sffn.gated_up_backward(dh, z, u, x, W1, W3, act="silu")
    dh[17] = math.nan
    got = sffn.gated_up_backward(dh, z, u, x, W1, W3, act="silu")
    assert torch.isnan(got[0][17]).all()
    rest = torch.arange(T, device=DEV) != 17
    assert torch.equal(got[0][rest], clean[0][rest])
    assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()  # a sum over the tokens


@pytest.mark.parametrize("T,D,H", [(300, 2560, 1024), (2048, 2560, 4100)])
def test_the_sign_of_a_kept_gate_is_the_sums(T, D, H):
    """z near 0 is computed again in fp32 (D / 64 steps a lane, their sum in 6 more): its sign is the exact sum's but where
    the exact sum is within that."""
    g = gen(36)
    x, W1, W3 = randn(g, T, D), randn(g, H, D) * D ** -0.5, randn(g, H, D) * D ** -0.5
    x[T // 2] = 0      # a padded token: exact zeros
    x[T // 3] *= 1e-9  # a token that is small as a whole
    W1[H // 2] = 0
    _, z, _ = sffn.gated_up_saved(x, W1, W3, act="relu")
    ref = x.double() @ W1.double().T
    S = x.double().abs() @ W1.double().abs().T
    assert (z[T // 2] == 0).all() and (z[:, H // 2] == 0).all()
    wrong = (z.double() * ref < 0) & (ref.abs() > (D / 64 + 8) * 2.0 ** -24 * S)
    wrong[T // 3] = False
    assert not wrong.any()
    close(z, ref, (D + 8) * 2.0 ** -23 * S)


def test_gated_no_tokens():
    W1, W3 = randn(gen(29), 24, 64).requires_grad_(), randn(gen(30), 24, 64).requires_grad_()
    x = torch.empty(0, 64, dtype=BF, device=DEV).requires_grad_()
    h = sffn.gated_up(x, W1, W3)
    assert h.shape == (0, 24)
    h.sum().backward()
    assert (W1.grad == 0).all() and (W3.grad == 0).all() and x.grad.shape == (0, 64)


@pytest.mark.parametrize("T", [2, 50])
def test_gated_strided_operands_and_result(T):
    g = gen(31)
    W1, W3 = randn(g, 72, 320), randn(g, 72, 320)
    x = randn(g, T, 400)[:, 40:360]
    y = sffn.gated_up(x, W1, W3)
    assert torch.equal(y, sffn.gated_up(x.contiguous(), W1, W3))
    out = torch.full((T + 2, 83), 5.0, dtype=BF, device=DEV)
    sffn.gated_up(x, W1, W3, out=out[:T, :72])
    assert torch.equal(out[:T, :72], y) and (out[T:] == 5).all() and (out[:, 72:] == 5).all()
    _, z, u = sffn.gated_up_saved(x, W1, W3)
    dh = randn(g, T, 90)[:, 3:75]  # neither aligned nor dense
    a = sffn.gated_up_backward(dh, z, u, x, W1, W3)
    b = sffn.gated_up_backward(dh.contiguous(), z, u, x.contiguous(), W1, W3)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_gated_repeats_its_bits():
    g = gen(32)
    x, W1, W3, dh = randn(g, 3000, 640), randn(g, 200, 640), randn(g, 200, 640), randn(g, 3000, 200)

    def step():
        h, z, u = sffn.gated_up_saved(x, W1, W3, act="silu")
        return (h, *sffn.gated_up_backward(dh, z, u, x, W1, W3, act="silu"))

    first = step()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, step()))


def test_calls_on_two_streams_at_once():
    g = gen(33)
    x, W1, W3, dh = randn(g, 500, 512), randn(g, 640, 512), randn(g, 640, 512), randn(g, 500, 640)
    q1, q3 = sffn.quantize_int4(W1), sffn.quantize_int4(W3)

    def both(stream):
        h, z, u = sffn.gated_up_saved(x, W1, W3, act="rsp", stream=stream)
        back = sffn.gated_up_backward(dh, z, u, x, W1, W3, act="rsp", stream=stream)
        return (h, *back, sffn.gated_up_int4(x, *q1, *q3, stream=stream), sffn.matmul_int4(x[:9], *q1, stream=stream))

    want = both(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [both(s) for _ in range(8) for s in streams]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_a_differentiable_call_on_another_stream():
    g = gen(34)
    x, W1, W3, dh = randn(g, 90, 128), randn(g, 64, 128), randn(g, 64, 128), randn(g, 90, 64)
    want = [t.clone().requires_grad_() for t in (x, W1, W3)]
    sffn.gated_up(*want).backward(dh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    have = [t.clone().requires_grad_() for t in (x, W1, W3)]
    side.wait_stream(torch.cuda.current_stream())
    h = sffn.gated_up(*have, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    h.backward(dh)  # the backward pass runs on the forward's stream, which autograd orders
    torch.cuda.synchronize()
    assert all(torch.equal(a.grad, b.grad) for a, b in zip(want, have))


def test_gated_rows_past_two_gigabytes():
    """Elements of h, z, u and of the gradients' operand pass 31 bits."""
    T, D, H = 280000, 8, 8192
    g = gen(35)
    x, W1, W3 = randn(g, T, D), randn(g, H, D), randn(g, H, D)
    h, z, u = sffn.gated_up_saved(x, W1, W3, act="relu")
    end = slice(T - 300, T)
    x64, a, b = x[end].double(), W1.double(), W3.double()
    dz, du = ((D + 8) * 2.0 ** -23 * (x64.abs() @ w.abs().T) for w in (a, b))
    check_h(h[end], x64 @ a.T, x64 @ b.T, dz, du, "relu")
    dh = torch.zeros_like(h)
    dh[end] = randn(g, 300, H)
    del h
    got = sffn.gated_up_backward(dh, z, u, x, W1, W3, act="relu")
    for y, (ref, bound) in zip((got[0][end], *got[1:]), grads(dh[end], z[end], u[end], x[end], W1, W3, "relu")):
        close(y, ref, bound)
    assert (got[0][:T - 300] == 0).all()


# ------------------------------------------------------------------ as they are used together


@pytest.mark.parametrize("T", [1, 20, 200])
def test_a_layer_is_trained_and_then_served_in_four_bits(T):
    """One step of a gated FFN by autograd against 64 bits, then the layer from 4-bit weights."""
    g = gen(40)
    D, H = 192, 256
    W1, W3, W2 = (randn(g, H, D) * D ** -0.5).requires_grad_(), (randn(g, H, D) * D ** -0.5).requires_grad_(), \
        (randn(g, D, H) * H ** -0.5).requires_grad_()
    x, dy = randn(g, T, D).requires_grad_(), randn(g, T, D)
    h = sffn.gated_up(x, W1, W3, act="silu")
    h.retain_grad()
    (h @ W2.T).backward(dy)
    dh = h.grad
    _, z, u = sffn.gated_up_saved(x.detach(), W1.detach(), W3.detach(), act="silu")
    for t, (ref, bound) in zip((x, W1, W3), grads(dh, z, u, x.detach(), W1.detach(), W3.detach(), "silu")):
        close(t.grad, ref, bound)
    with torch.no_grad():
        for w in (W1, W3, W2):
            w -= 0.1 * w.grad
    ffn = sffn.Int4FFN(W1.detach(), W3.detach(), W2.detach(), act="silu")
    x = x.detach()
    y = ffn(x)
    q1, q3, q2 = meant(*ffn.w1, 64), meant(*ffn.w3, 64), meant(*ffn.w2, None)
    h64 = product(x.double() @ q1.T, x.double() @ q3.T, "silu")
    hb = sffn.gated_up_int4(x, *ffn.w1, *ffn.w3, act="silu")
    check_h(hb, x.double() @ q1.T, x.double() @ q3.T, bound4(x, q1, T > ROWS, True), bound4(x, q3, T > ROWS, True), "silu")
    close(y, hb.double() @ q2.T, bound4(hb, q2, T > ROWS, False))
    assert ((y.double() - h64 @ q2.T).norm() / (h64 @ q2.T).norm()).item() < 3 * 2.0 ** -8  # three roundings to bf16


def test_the_layer_holds_an_int4_handles_codes():
    """Int4FFN's codes are those that an int4 handle makes of the same weights."""
    g = gen(41)
    D, H = 256, 320
    W1, W3, W2 = randn(g, H, D), randn(g, H, D), randn(g, D, H)
    layer = sffn.Int4FFN(W1, W3, W2)
    handle = sffn.SparseFFN(D, H, 0, "relu", "int4")
    handle.set_weights(W1, None, W3, W2)
    q1, s1, q3, s3, q2, s2 = handle.int8_weights()
    assert torch.equal(unpack(layer.w1[0]), q1) and torch.equal(layer.w1[1], s1)
    assert torch.equal(unpack(layer.w3[0]), q3) and torch.equal(layer.w3[1], s3)
    assert torch.equal(unpack(layer.w2[0]), q2) and torch.equal(layer.w2[1][:, 0], s2)
    x = randn(g, 1, D)
    y, z = layer(x).double(), handle(x).double()
    assert ((y - z).norm() / z.norm()).item() < 3 * 2.0 ** -8  # both results are rounded, and the layer's h
    handle.close()


def test_long_products_follow_one_another_without_a_stop():
    """Pair tiles launched into the end of the kernel that makes their weights, some thousand times."""
    g = gen(42)
    sets = [(weights4(g, 14336, 4096, 64), randn(g, 2048, 4096)) for _ in range(3)]
    first = [sffn.matmul_int4(x, *w) for w, x in sets]
    torch.cuda.synchronize()
    for n in range(500):
        got = [sffn.matmul_int4(x, *w) for w, x in sets]
        if n % 50 == 49:
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(first, got))
