"""The mixture-of-experts and 8-bit operators against plain implementations in 64 bits.

Tolerances count roundings: a result rounded to type t is off by eps(t) / 2 of itself, and an fp32
sum of K products by at most K * 2^-23 of the sum of their magnitudes (each step one rounding, or
one truncation on the tensor cores).
"""
import math

import pytest

torch = pytest.importorskip("torch")
import activation_sparse_gated_gb300 as sffn  # noqa: E402

pytestmark = pytest.mark.gpu
BF, DEV = torch.bfloat16, "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def no_device_error(cuda_ok):
    yield
    sffn.sffn_check()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def close(y, ref, bound):
    """|y - ref| <= bound + half a step of y's type, everywhere; NaN and infinities in the same places."""
    y64 = y.double()
    assert torch.equal(torch.isnan(y64), torch.isnan(ref))
    ok = torch.isfinite(ref)
    off = (y64 - ref).abs() - HALF[y.dtype] * 1.01 * ref.abs() - bound
    worst = off[ok].max().item() if ok.any() else 0.0
    assert worst <= 1e-30, f"off by {worst} more than the bound"


# ------------------------------------------------------------------ route


def plain_route(z, k, score, normalize):
    z = z.double().cpu()
    T, E = z.shape
    z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    order = torch.sort(-z, dim=1, stable=True).indices[:, :k]  # equal values keep the order of their indices
    v = z.gather(1, order)
    is_open = v > -math.inf
    m = torch.where(is_open[:, :1], v[:, :1], torch.zeros_like(v[:, :1]))
    ex = lambda a: torch.where(a == m, torch.ones_like(a), torch.exp(a - m))  # noqa: E731
    w = ex(v) if score == "softmax" else torch.sigmoid(v)
    w = torch.where(is_open, w, torch.zeros_like(w))
    if normalize:
        total = w.sum(1, keepdim=True)
    else:
        total = torch.where(z > -math.inf, ex(z), torch.zeros_like(z)).sum(1, keepdim=True)
        total = total if score == "softmax" else torch.ones_like(total)
    w = torch.where(total > 0, w / total, torch.zeros_like(w))
    ids = torch.where(is_open, order, torch.full_like(order, -1))
    flat = ids.reshape(-1)
    groups = [torch.nonzero(flat == e).reshape(-1).tolist() for e in range(E)]
    rows, offsets = sum(groups, []), [0]
    for part in groups:
        offsets.append(offsets[-1] + len(part))
    return w, ids, offsets, rows + [-1] * (T * k - len(rows))


def check_route(z, k, score, normalize):
    w, ids, offsets, rows = sffn.route(z, k, score=score, normalize=normalize)
    pw, pids, poff, prows = plain_route(z, k, score, normalize)
    assert torch.equal(ids.cpu().long(), pids)
    assert offsets.tolist() == poff
    assert rows.tolist() == prows
    # exp (2 ulp of its own and the rounded difference), a sum of E terms, a quotient
    tol = (z.shape[1] + 8) * 2.0 ** -23
    torch.testing.assert_close(w.double().cpu(), pw, rtol=tol, atol=1e-30 if score == "softmax" else 1e-37)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 7, 7), (17, 33, 4), (128, 64, 8), (255, 256, 8),
                                   (257, 8, 8), (300, 100, 32), (513, 1024, 5), (2049, 16, 1), (1000, 96, 3)])
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_sizes(T, E, k, score, normalize):
    check_route(torch.randn(T, E, generator=gen(T + E), device=DEV), k, score, normalize)


@pytest.mark.parametrize("T", [5, 700])
def test_route_ties_masks_and_odd_values(T):
    z = torch.randn(T, 48, generator=gen(1), device=DEV).round()  # many ties, zeros of both signs among them
    z[0] = -math.inf                 # a token with no expert
    z[1] = math.nan
    z[2] = 0.0
    z[3, 5] = math.inf
    z[3, 9] = math.inf
    z[4] = torch.finfo(torch.float32).min
    z[4, 7] = math.nan
    for score in ("softmax", "sigmoid"):
        check_route(z, 6, score, True)
    check_route(z.to(BF), 6, "softmax", True)


def test_route_negative_zero_ties_with_zero():
    z = torch.full((1, 8), -1.0, device=DEV)
    z[0, 2], z[0, 5] = -0.0, 0.0
    assert sffn.route(z, 2).ids.tolist() == [[2, 5]]


def test_route_strided_logits_and_empty():
    z = torch.randn(300, 96, generator=gen(2), device=DEV)
    a, b = sffn.route(z[:, :64], 8), sffn.route(z[:, :64].contiguous(), 8)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    empty = sffn.route(z[:0], 8)
    assert empty.offsets.tolist() == [0] * 97 and empty.ids.shape == (0, 8)


# ------------------------------------------------------------------ quantize


@pytest.mark.parametrize("T,K", [(1, 1), (1, 2560), (3, 17), (64, 384), (5, 1000), (33, 1024), (7, 4096), (9, 8200),
                                 (4, 14336), (2, 20000), (3, 65536)])
def test_quantize_tokens(T, K):
    x = torch.randn(T, K, generator=gen(K), device=DEV).to(BF)
    if T > 1:
        x[1] = 0
    if T > 2:
        x[2] = x[2] * 1e30
    q, s = sffn.quantize_tokens(x)
    xc = x.float().cpu().numpy()
    sc = abs(xc).max(1) / xc.dtype.type(127)
    code = (xc / (sc + (sc == 0))[:, None]).round().clip(-127, 127)
    assert (s.cpu().numpy() == sc).all()
    assert (q.cpu().numpy() == code).all()


@pytest.mark.parametrize("T", [1, 2, 9, 700])
@pytest.mark.parametrize("K,pad", [(1, 0), (3, 0), (7, 8), (9, 0), (15, 16), (1001, 0), (1019, 8), (2047, 0), (4095, 5),
                                   (8193, 0), (8196, 64), (11577, 0), (16370, 0), (16383, 0), (16384, 0)])
def test_quantize_rows_that_start_anywhere(T, K, pad):
    """Rows of odd lengths next to rows of NaN and infinities, which must not reach them, and codes next to codes."""
    wide = torch.randn(T, K + pad, generator=gen(T + K), device=DEV).to(BF)
    x = wide[:, :K]
    wide[:, K:] = math.inf
    for r, v in ((1, math.nan), (4, math.inf), (6, 0.0)):
        x[r:r + 1] = v
    q, s = sffn.quantize_tokens(x)
    for r in range(T):
        if r in (1, 4):
            assert torch.isnan(s[r]) and (q[r] == 0).all()
    xc = x.float().cpu().numpy()
    xc[[r for r in (1, 4) if r < T]] = 0
    sc = abs(xc).max(1) / xc.dtype.type(127)
    code = (xc / (sc + (sc == 0))[:, None]).round().clip(-127, 127)
    assert (torch.nan_to_num(s).cpu().numpy() == sc).all()
    assert (q.cpu().numpy() == code).all()


def test_quantize_special_values_and_strides():
    x = torch.randn(6, 512, generator=gen(3), device=DEV).to(BF)
    x[1, 3], x[2, 5], x[3, 7] = math.nan, math.inf, -math.inf
    x[4] = 1e-40  # below the smallest normal value
    q, s = sffn.quantize_tokens(x)
    assert torch.isnan(s[1:4]).all() and (q[1:4] == 0).all()
    assert torch.isfinite(s[[0, 4, 5]]).all()
    big = torch.randn(5, 300, generator=gen(4), device=DEV).to(BF)
    for view in (big[:, 3:203], big[:, 8:264], big[::2]):
        a, b = sffn.quantize_tokens(view), sffn.quantize_tokens(view.contiguous())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ products


def int8_operands(g, rows, K, full=False):
    q = torch.randint(-128 if full else -127, 128, (rows, K), generator=g, device=DEV, dtype=torch.int8)
    return q, torch.rand(rows, generator=g, device=DEV) + 0.5


def int8_bound(xq, wq, scale):
    """fp32 holds the integer sums below 2^24; past it each step may lose 2^-23 of the magnitudes."""
    mag = xq.double().abs() @ wq.double().abs().T
    return torch.where(mag < 2 ** 24, torch.zeros_like(mag), mag * xq.shape[1] * 2.0 ** -23) * scale


@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 7168, 2560), (2, 129, 64), (3, 100, 400), (8, 1024, 384),
                                   (9, 257, 1040), (16, 2560, 512), (17, 128, 128), (31, 300, 2560), (77, 2560, 7168),
                                   (64, 1000, 4096), (128, 128, 144), (129, 513, 640), (257, 384, 1024),
                                   (500, 1001, 272), (1030, 520, 2048), (40, 90, 65536)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_int8(T, N, K, out):
    g = gen(T * 7 + N)
    xq, sx = int8_operands(g, T, K, full=True)
    wq, sw = int8_operands(g, N, K)
    y = sffn.matmul_int8(xq, sx, wq, sw, dtype=out)
    scale = torch.outer(sx.double(), sw.double())
    ref = (xq.double() @ wq.double().T) * scale
    close(y, ref, 3 * 2.0 ** -24 * ref.abs() + int8_bound(xq, wq, scale))


@pytest.mark.parametrize("T,N", [(700, 4001), (800, 4000), (310, 9000)])
@pytest.mark.parametrize("K", [16, 144, 272, 448, 1104])
def test_matmul_int8_several_tiles_a_block(T, N, K):
    """More tiles than blocks, each of an odd or even number of stages: the stages' phases run on from tile to tile."""
    test_matmul_int8(T, N, K, "bf16")
    test_matmul_int8(T, N, K, "f32")


def test_matmul_int8_strides_zero_scales_and_out():
    g = gen(11)
    big, sx = int8_operands(g, 40, 512)
    wq, sw = int8_operands(g, 70, 256)
    sx[3], sx[5] = 0.0, math.nan
    x = big[:, 128:384]
    y = sffn.matmul_int8(x, sx, wq, sw, dtype="f32")
    ref = (x.double() @ wq.double().T) * torch.outer(sx.double(), sw.double())
    close(y, ref, 3 * 2.0 ** -24 * ref.abs())
    assert (y[3] == 0).all() and torch.isnan(y[5]).all()
    wide = torch.full((40, 100), 7.0, device=DEV)
    sffn.matmul_int8(x, sx, wq, sw, out=wide[:, 10:80])
    assert torch.equal(wide[:, 10:80].nan_to_num(), y.nan_to_num())
    assert (wide[:, :10] == 7).all() and (wide[:, 80:] == 7).all()


def offsets_of(counts):
    return torch.tensor([0] + counts, device=DEV).cumsum(0).to(torch.int32)


GROUPS = [[1], [0, 1, 0], [1, 1, 1, 1], [3, 0, 5, 1], [16, 17, 0, 31, 1], [0, 0, 40, 0], [130, 1, 0, 127],
          [300, 5, 129, 256, 257, 0, 2], [0] * 30 + [2, 1] + [0] * 30 + [9]]


@pytest.mark.parametrize("counts", GROUPS, ids=str)
@pytest.mark.parametrize("N,K", [(1, 8), (100, 72), (128, 64), (256, 384), (1000, 520)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_grouped_matmul_bf16(counts, N, K, out):
    g, R, E = gen(N + K), sum(counts), len(counts)
    x = torch.randn(R, K, generator=g, device=DEV).to(BF)
    w = torch.randn(E, N, K, generator=g, device=DEV).to(BF)
    off = offsets_of(counts)
    y = sffn.grouped_matmul(x, w, off, dtype=out)
    b = off.tolist()
    for e in range(E):
        xe, we = x[b[e]:b[e + 1]].double(), w[e].double()
        close(y[b[e]:b[e + 1]], xe @ we.T, K * 2.0 ** -23 * (xe.abs() @ we.abs().T))


@pytest.mark.parametrize("counts", GROUPS, ids=str)
@pytest.mark.parametrize("N,K", [(8, 8), (104, 70), (128, 64), (256, 384), (1000, 519)])
def test_grouped_matmul_transposed_weights(counts, N, K):
    g, R, E = gen(N + K), sum(counts), len(counts)
    pitch = (K + 7) // 8 * 8
    x = torch.zeros(R, pitch, device=DEV, dtype=BF)
    x[:, :K] = torch.randn(R, K, generator=g, device=DEV).to(BF)
    w = torch.zeros(E, pitch, N, device=DEV, dtype=BF)
    w[:, :K] = torch.randn(E, K, N, generator=g, device=DEV).to(BF)
    off = offsets_of(counts)
    y = sffn.grouped_matmul(x, w, off, transposed=True)
    b = off.tolist()
    for e in range(E):
        xe, we = x[b[e]:b[e + 1]].double(), w[e].double()
        close(y[b[e]:b[e + 1]], xe @ we, K * 2.0 ** -23 * (xe.abs() @ we.abs()))


@pytest.mark.parametrize("counts", GROUPS, ids=str)
@pytest.mark.parametrize("N,K", [(1, 16), (100, 80), (256, 384), (1000, 528)])
def test_grouped_matmul_int8(counts, N, K):
    g, R, E = gen(N + K), sum(counts), len(counts)
    x, sx = int8_operands(g, R, K)
    w, sw = int8_operands(g, E * N, K, full=True)
    w, sw = w.view(E, N, K), sw.view(E, N)
    off = offsets_of(counts)
    y = sffn.grouped_matmul(x, w, off, sx=sx, sw=sw, dtype="f32")
    b = off.tolist()
    for e in range(E):
        r = slice(b[e], b[e + 1])
        scale = torch.outer(sx[r].double(), sw[e].double())
        ref = (x[r].double() @ w[e].double().T) * scale
        close(y[r], ref, 3 * 2.0 ** -24 * ref.abs() + int8_bound(x[r], w[e], scale))


@pytest.mark.parametrize("T,k", [(3, 2), (50, 3), (300, 2)])
def test_grouped_matmul_reads_tokens_through_an_index(T, k):
    g, E, N, K = gen(T), 5, 200, 136
    routing = sffn.route(torch.randn(T, E, generator=g, device=DEV), k)
    big = torch.randn(T, K + 24, generator=g, device=DEV).to(BF)
    x = big[:, 8:8 + K]
    w = torch.randn(E, N, K, generator=g, device=DEV).to(BF)
    y = sffn.grouped_matmul(x, w, routing.offsets, index=routing.rows, index_div=k, dtype="f32")
    z = sffn.grouped_matmul(x[(routing.rows // k).long()].contiguous(), w, routing.offsets, dtype="f32")
    assert torch.equal(y, z)


def test_grouped_matmul_int8_reads_tokens_through_an_index():
    g, T, k, E, N, K = gen(61), 120, 3, 5, 200, 144
    routing = sffn.route(torch.randn(T, E, generator=g, device=DEV), k)
    x, sx = int8_operands(g, T, K)
    w, sw = int8_operands(g, E * N, K)
    w, sw = w.view(E, N, K), sw.view(E, N)
    src = (routing.rows // k).long()
    y = sffn.grouped_matmul(x, w, routing.offsets, sx=sx, sw=sw, index=routing.rows, index_div=k, dtype="f32")
    z = sffn.grouped_matmul(x[src].contiguous(), w, routing.offsets, sx=sx[src].contiguous(), sw=sw, dtype="f32")
    assert torch.equal(y, z)


@pytest.mark.parametrize("T,N,K", [(2048, 2048, 4096), (2100, 3001, 2064), (3000, 5001, 1040)])
def test_matmul_int8_copies(T, N, K):
    """Enough tiles for the fp16 copies of the codes."""
    test_matmul_int8(T, N, K, "bf16")
    test_matmul_int8(T, N, K, "f32")


@pytest.mark.parametrize("k,index", [(1, False), (2, True)])
def test_grouped_matmul_int8_copies(k, index):
    g, T, E, N, K = gen(63), 1800 // k, 2, 6000, 2064
    R, rows = T * k, torch.randperm(T * k, generator=torch.Generator().manual_seed(3)).to(DEV, torch.int32)
    x, sx = int8_operands(g, T if index else R, K, full=True)
    w, sw = int8_operands(g, E * N, K)
    offsets = torch.tensor([0, R // 3, R], dtype=torch.int32, device=DEV)
    y = sffn.grouped_matmul(x, w.view(E, N, K), offsets, sx, sw.view(E, N), index=rows if index else None,
                            index_div=k, dtype="f32")
    src = (rows // k).long() if index else torch.arange(R, device=DEV)
    xq, s = x[src], sx[src]
    for e, (a, b) in enumerate(((0, R // 3), (R // 3, R))):
        scale = torch.outer(s[a:b].double(), sw.view(E, N)[e].double())
        ref = (xq[a:b].double() @ w.view(E, N, K)[e].double().T) * scale
        close(y[a:b], ref, 3 * 2.0 ** -24 * ref.abs() + int8_bound(xq[a:b], w.view(E, N, K)[e], scale))


def test_grouped_matmul_int8_long_groups():
    """Groups long enough for the fp16 copies of the codes, strided rows, with and without an index."""
    g, T, k, E, N, K = gen(62), 1300, 2, 3, 264, 400
    routing = sffn.route(torch.randn(T, E, generator=g, device=DEV), k)
    big, sx = int8_operands(g, T, K + 48, full=True)
    x = big[:, 32:32 + K]
    w, sw = int8_operands(g, E * N, K)
    w, sw = w.view(E, N, K), sw.view(E, N)
    assert sffn.sffn_grouped_workspace(T * k, T, N, K, E, sffn.SFFN_I8) > 0
    src = (routing.rows // k).long()
    y = sffn.grouped_matmul(x, w, routing.offsets, sx=sx, sw=sw, index=routing.rows, index_div=k, dtype="f32")
    z = sffn.grouped_matmul(x[src].contiguous(), w, routing.offsets, sx=sx[src].contiguous(), sw=sw, dtype="f32")
    assert torch.equal(y, z)
    b = routing.offsets.tolist()
    for e in range(E):
        r = slice(b[e], b[e + 1])
        xe = x[src[r]]
        scale = torch.outer(sx[src[r]].double(), sw[e].double())
        ref = (xe.double() @ w[e].double().T) * scale
        close(y[r], ref, 3 * 2.0 ** -24 * ref.abs() + int8_bound(xe, w[e], scale))


@pytest.mark.parametrize("counts", [[20, 0, 33], [130], [17, 64, 300]], ids=str)
@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_matmul_few_tiles_long_sums(counts, transposed):
    """Few tiles and a long sum: blocks of a cluster cut K between them."""
    g, R, E, N, K = gen(71), sum(counts), len(counts), 264, 3000
    x = torch.randn(R, K, generator=g, device=DEV).to(BF)
    w = torch.randn(E, N, K, generator=g, device=DEV).to(BF)
    off = offsets_of(counts)
    y = sffn.grouped_matmul(x, w.transpose(1, 2).contiguous() if transposed else w, off, transposed=transposed, dtype="f32")
    z = sffn.grouped_matmul(x, w.transpose(1, 2).contiguous() if transposed else w, off, transposed=transposed, dtype="f32")
    assert torch.equal(y, z)
    b = off.tolist()
    for e in range(E):
        xe, we = x[b[e]:b[e + 1]].double(), w[e].double()
        close(y[b[e]:b[e + 1]], xe @ we.T, K * 2.0 ** -23 * (xe.abs() @ we.abs().T))


PAIRS = [130, 97, 256, 1, 0, 300, 64, 257, 100, 128, 200, 31, 180, 96, 0, 513, 140, 33, 128, 160]


@pytest.mark.parametrize("N,K,out", [(1000, 136, "bf16"), (1001, 72, "f32"), (1003, 200, "bf16"), (2056, 64, "f32")])
@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_matmul_long_ragged_groups(N, K, out, transposed):
    """Groups long and many enough for tiles of a pair of blocks; odd widths take narrow stores."""
    if transposed:
        N = N // 8 * 8
    g, R, E = gen(N), sum(PAIRS), len(PAIRS)
    x = torch.randn(R, K, generator=g, device=DEV).to(BF)
    w = torch.randn(E, N, K, generator=g, device=DEV).to(BF)
    off = offsets_of(PAIRS)
    wide = torch.full((R, N + 5), 3.0, device=DEV, dtype=BF if out == "bf16" else torch.float32)
    y = sffn.grouped_matmul(x, w.transpose(1, 2).contiguous() if transposed else w, off, transposed=transposed,
                            out=wide[:, 3:3 + N])
    z = sffn.grouped_matmul(x, w.transpose(1, 2).contiguous() if transposed else w, off, transposed=transposed, dtype=out)
    assert torch.equal(y, z)
    assert (wide[:, :3] == 3).all() and (wide[:, 3 + N:] == 3).all()
    b = off.tolist()
    for e in range(E):
        xe, we = x[b[e]:b[e + 1]].double(), w[e].double()
        close(y[b[e]:b[e + 1]], xe @ we.T, K * 2.0 ** -23 * (xe.abs() @ we.abs().T))


def test_grouped_matmul_long_groups_read_tokens_through_an_index():
    g, T, k, E, N, K = gen(72), 1400, 2, 20, 1000, 136
    routing = sffn.route(torch.randn(T, E, generator=g, device=DEV), k)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    w = torch.randn(E, N, K, generator=g, device=DEV).to(BF)
    y = sffn.grouped_matmul(x, w, routing.offsets, index=routing.rows, index_div=k, dtype="f32")
    z = sffn.grouped_matmul(x[(routing.rows // k).long()].contiguous(), w, routing.offsets, dtype="f32")
    assert torch.equal(y, z)


@pytest.mark.parametrize("counts", [[3, 0, 1, 2], [1] * 30, [0, 4], [2]], ids=str)
@pytest.mark.parametrize("N,K", [(33, 48), (400, 1040), (6000, 256)])
def test_grouped_matmul_int8_few_rows(counts, N, K):
    """Groups of one to four rows: the dot products of four."""
    g, R, E = gen(N + K), sum(counts), len(counts)
    x, sx = int8_operands(g, R, K, full=True)
    w, sw = int8_operands(g, E * N, K, full=True)
    w, sw = w.view(E, N, K), sw.view(E, N)
    off = offsets_of(counts)
    y = sffn.grouped_matmul(x, w, off, sx=sx, sw=sw, dtype="f32")
    b = off.tolist()
    for e in range(E):
        r = slice(b[e], b[e + 1])
        scale = torch.outer(sx[r].double(), sw[e].double())
        ref = (x[r].double() @ w[e].double().T) * scale
        close(y[r], ref, 3 * 2.0 ** -24 * ref.abs() + int8_bound(x[r], w[e], scale))


def test_grouped_matmul_past_32_bits():
    """Weights, rows and results whose byte and element offsets pass 32 bits."""
    g = gen(81)
    E, N, K = 40, 7168, 8000  # 2.3e9 weights
    w = torch.zeros(E, N, K, device=DEV, dtype=BF)
    w[-1] = torch.randn(N, K, generator=g, device=DEV).to(BF)
    x = torch.randn(20, K, generator=g, device=DEV).to(BF)
    y = sffn.grouped_matmul(x, w, offsets_of([0] * (E - 1) + [20]), dtype="f32")
    xe, we = x.double(), w[-1].double()
    close(y, xe @ we.T, K * 2.0 ** -23 * (xe.abs() @ we.abs().T))
    del w, we
    R, N, K = 310000, 7168, 64  # 2.2e9 results
    x = torch.randn(R, K, generator=g, device=DEV).to(BF)
    w = torch.randn(1, N, K, generator=g, device=DEV).to(BF)
    y = sffn.grouped_matmul(x, w, offsets_of([R]))
    for r in (slice(0, 50), slice(R - 300, R)):
        xe, we = x[r].double(), w[0].double()
        close(y[r], xe @ we.T, K * 2.0 ** -23 * (xe.abs() @ we.abs().T))


def test_two_streams_at_once():
    """Calls that overlap on the GPU share nothing."""
    g, E, N, K = gen(83), 6, 520, 512
    x = torch.randn(600, K, generator=g, device=DEV).to(BF)
    w = torch.randn(E, N, K, generator=g, device=DEV).to(BF)
    q, sx = int8_operands(g, 600, K)
    wq, sw = int8_operands(g, N, K)
    off = offsets_of([100] * 6)
    want = sffn.grouped_matmul(x, w, off), sffn.matmul_int8(q, sx, wq, sw), sffn.route(x[:, :64].float(), 4)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        got.append((sffn.grouped_matmul(x, w, off, stream=a), sffn.matmul_int8(q, sx, wq, sw, stream=b),
                    sffn.route(x[:, :64].float(), 4, stream=b)))
    torch.cuda.synchronize()
    for y, z, r in got:
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])
        assert all(torch.equal(p, v) for p, v in zip(r, want[2]))


@pytest.mark.parametrize("E", [200, 1000])
def test_grouped_matmul_many_experts(E):
    """Tables of many groups, most of them empty or short."""
    g, N, K = gen(E), 136, 160
    counts = torch.randint(0, 24, (E,), generator=torch.Generator().manual_seed(E)).tolist()
    off = offsets_of(counts)
    R, b = sum(counts), off.tolist()
    x = torch.randn(R, K, generator=g, device=DEV).to(BF)
    w = torch.randn(E, N, K, generator=g, device=DEV).to(BF)
    q, sx = int8_operands(g, R, K)
    wq, sw = int8_operands(g, E * N, K)
    wq, sw = wq.view(E, N, K), sw.view(E, N)
    y = sffn.grouped_matmul(x, w, off, dtype="f32")
    z = sffn.grouped_matmul(q, wq, off, sx=sx, sw=sw, dtype="f32")
    for e in range(0, E, 7):
        r = slice(b[e], b[e + 1])
        xe, we = x[r].double(), w[e].double()
        close(y[r], xe @ we.T, K * 2.0 ** -23 * (xe.abs() @ we.abs().T))
        scale = torch.outer(sx[r].double(), sw[e].double())
        ref = (q[r].double() @ wq[e].double().T) * scale
        close(z[r], ref, 3 * 2.0 ** -24 * ref.abs() + int8_bound(q[r], wq[e], scale))


def test_grouped_matmul_source_rows_out_of_range_read_as_zeros():
    g = gen(21)
    x = torch.randn(10, 64, generator=g, device=DEV).to(BF)
    w = torch.randn(2, 128, 64, generator=g, device=DEV).to(BF)
    for n in (4, 40):
        index = torch.arange(n, dtype=torch.int32, device=DEV) % 10
        index[1], index[2] = 10, -7
        y = sffn.grouped_matmul(x, w, offsets_of([n // 2, n - n // 2]), index=index, dtype="f32")
        assert (y[1:3] == 0).all()
        assert (y[0] != 0).any() and torch.isfinite(y).all()


@pytest.mark.parametrize("n", [6, 200])
def test_grouped_matmul_keeps_rows_past_the_groups(n):
    g = gen(22)
    x = torch.randn(n, 64, generator=g, device=DEV).to(BF)
    x[n // 2:] = math.nan  # rows of no group
    w = torch.randn(3, 96, 64, generator=g, device=DEV).to(BF)
    y = torch.full((n, 96), 5.0, device=DEV)
    sffn.grouped_matmul(x, w, offsets_of([1, 0, n // 2 - 1]), out=y)
    assert torch.isfinite(y).all() and (y[n // 2:] == 5).all()
    # a broken list of offsets stays inside the buffers: cut to R, never below the group's start
    guard = torch.full((n + 4, 96), 5.0, device=DEV)
    bad = torch.tensor([0, n + 50, -3, 2 * n], dtype=torch.int32, device=DEV)
    sffn.grouped_matmul(x, w, bad, out=guard[2:n + 2])
    assert (guard[:2] == 5).all() and (guard[n + 2:] == 5).all()


def test_grouped_matmul_keeps_nan_and_infinity_to_their_rows():
    g = gen(23)
    for n in (4, 60):
        x = torch.randn(2 * n, 128, generator=g, device=DEV).to(BF)
        w = torch.randn(2, 72, 128, generator=g, device=DEV).to(BF)
        clean = sffn.grouped_matmul(x, w, offsets_of([n, n]))
        x[1, 5], x[n, 7] = math.nan, math.inf
        y = sffn.grouped_matmul(x, w, offsets_of([n, n]))
        keep = [r for r in range(2 * n) if r not in (1, n)]
        assert torch.equal(y[keep], clean[keep])
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[n]).any()


# ------------------------------------------------------------------ the experts


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    v = z * torch.sigmoid(z)
    return v if act == "silu" else torch.where(z > 0, v, torch.zeros_like(v))


def check_experts(x, routing, W1, W3, W2t, act, y):
    """Against 64 bits.  h may be off by the fp32 sums of its two factors and one rounding to bf16; a choice's
    product by its sum; the combination by k sums."""
    T, D = x.shape
    k, E, H = routing.ids.shape[1], W1.shape[0], W1.shape[1]
    ref, bound = torch.zeros(T, D, dtype=torch.float64, device=DEV), torch.zeros(T, D, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = torch.nonzero(routing.ids == e, as_tuple=True)
        if not len(t):
            continue
        xe, w1, w3, w2 = x[t].double(), W1[e].double(), W3[e].double(), W2t[e].double()
        z, u = xe @ w1.T, xe @ w3.T
        a = act64(z, act)
        dz, du = (D * 2.0 ** -23 * (xe.abs() @ w.abs().T) for w in (w1, w3))
        h = a * u
        dh = 1.1 * dz * u.abs() + (a.abs() + 1.1 * dz) * du + 2.0 ** -8 * 1.01 * h.abs() + 2.0 ** -20 * h.abs()
        w = routing.weights[t, j].double()[:, None]
        mag = h.abs() @ w2.abs()
        ref.index_add_(0, t, w * (h @ w2))
        bound.index_add_(0, t, w * (dh @ w2.abs() + (H + k + 4) * 2.0 ** -23 * mag))
    close(y, ref, bound)


@pytest.mark.parametrize("T,E,k,D,H", [(1, 1, 1, 8, 1), (1, 8, 2, 128, 100), (1, 64, 8, 2560, 1024), (2, 4, 3, 264, 65), (1, 4, 2, 22000, 20), (3, 4, 2, 6000, 24),
                                       (5, 16, 4, 384, 130), (33, 8, 2, 520, 200), (64, 64, 8, 256, 96),
                                       (20, 2, 2, 136, 90), (2, 8, 8, 64, 2600), (200, 6, 2, 384, 257), (513, 5, 3, 256, 128), (300, 128, 4, 136, 72), (40, 4, 2, 2048, 200), (24, 2, 2, 256, 4000), (700, 4, 2, 200, 300), (130, 1, 1, 512, 1000)])
@pytest.mark.parametrize("act", ["relu", "rsp", "silu"])
def test_experts_forward(T, E, k, D, H, act):
    g = gen(T + D + H)
    x = torch.randn(T, D, generator=g, device=DEV).to(BF)
    W1, W3 = ((torch.randn(E, H, D, generator=g, device=DEV) * D ** -0.5).to(BF) for _ in range(2))
    W2t = (torch.randn(E, H, D, generator=g, device=DEV) * H ** -0.5).to(BF)
    x[:, -1] = 1
    W1[:, :, -1] = -1.0
    routing = sffn.route(torch.randn(T, E, generator=g, device=DEV), k)
    y = sffn.experts_forward(x, routing, W1, W3, W2t, act=act)
    check_experts(x, routing, W1, W3, W2t, act, y)
    again = sffn.experts_forward(x, routing, W1, W3, W2t, act=act)
    assert torch.equal(y, again)


@pytest.mark.parametrize("T", [3, 90])
def test_experts_closed_tokens_strides_and_streams(T):
    g, E, k, D, H = gen(T), 6, 2, 256, 96
    big = torch.randn(T, 2 * D, generator=g, device=DEV).to(BF)
    x = big[:, D // 2:D // 2 + D]
    W1, W3, W2t = ((torch.randn(E, H, D, generator=g, device=DEV) * 0.1).to(BF) for _ in range(3))
    z = torch.randn(T, E, generator=g, device=DEV)
    z[1] = -math.inf                        # no expert at all
    z[2, :] = -math.inf
    z[2, 3] = 0.5                           # one expert for two places
    z[:, 5] = -math.inf                     # an expert that nobody takes
    routing = sffn.route(z, k)
    y = sffn.experts_forward(x, routing, W1, W3, W2t)
    assert (y[1] == 0).all()
    check_experts(x.contiguous(), routing, W1, W3, W2t, "relu", y)
    assert torch.equal(sffn.experts_forward(x, tuple(routing), W1, W3, W2t), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r2 = sffn.route(z, k, stream=side)
    y2 = sffn.experts_forward(x, r2, W1, W3, W2t, stream=side)
    side.synchronize()
    assert torch.equal(y, y2)


def test_experts_many_tokens():
    """More tokens than a grid's second dimension holds."""
    g, T, E, k, D, H = gen(33), 70000, 3, 2, 64, 40
    x = torch.randn(T, D, generator=g, device=DEV).to(BF)
    W1, W3, W2t = ((torch.randn(E, H, D, generator=g, device=DEV) * 0.2).to(BF) for _ in range(3))
    routing = sffn.route(torch.randn(T, E, generator=g, device=DEV), k)
    check_experts(x, routing, W1, W3, W2t, "silu", sffn.experts_forward(x, routing, W1, W3, W2t, act="silu"))


def test_moe_layer_and_graph_capture():
    g, T, E, k, D, H = gen(31), 40, 8, 2, 256, 160
    x = torch.randn(T, D, generator=g, device=DEV).to(BF)
    Wr = torch.randn(E, D, generator=g, device=DEV)
    W1, W3 = ((torch.randn(E, H, D, generator=g, device=DEV) * 0.1).to(BF) for _ in range(2))
    W2 = (torch.randn(E, D, H, generator=g, device=DEV) * 0.1).to(BF)
    moe = sffn.MoEFFN(Wr, W1, W3, W2, k, act="rsp")
    y = moe(x)
    check_experts(x, moe.route(x), W1, W3, W2.transpose(1, 2), "rsp", y)
    for n in (1, T):
        xs, z = x[:n].clone(), torch.randn(n, E, generator=g, device=DEV)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            sffn.experts_forward(xs, sffn.route(z, k), moe.W1, moe.W3, moe.W2t)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = sffn.experts_forward(xs, sffn.route(z, k), moe.W1, moe.W3, moe.W2t)
        for _ in range(2):
            z.copy_(torch.randn(n, E, generator=g, device=DEV))
            xs.copy_(xs.flip(0))
            graph.replay()
            want = sffn.experts_forward(xs, sffn.route(z, k), moe.W1, moe.W3, moe.W2t)
            assert torch.equal(out, want)


def test_int8_linear_of_quantised_tokens():
    """The two int8 operators as a served linear layer uses them."""
    g, T, N, K = gen(41), 50, 384, 1024
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    w = torch.randn(N, K, generator=g, device=DEV).to(BF)
    wq, sw = sffn.quantize_tokens(w)  # the same rule gives one scale per output channel
    xq, sx = sffn.quantize_tokens(x)
    y = sffn.matmul_int8(xq, sx, wq, sw)
    ref = x.double() @ w.double().T
    # half a code step on either side of every product
    bound = (sx.double()[:, None] / 2 * 1.001) * w.double().abs().sum(1) + \
        x.double().abs().sum(1)[:, None] * (sw.double() / 2 * 1.001) + K * torch.outer(sx.double(), sw.double()) / 4
    close(y, ref, bound * (1 + 2.0 ** -7))


def test_calls_with_and_without_the_native_module(monkeypatch):
    """The calls' one-step form and the wrappers' own give the same results and take the same cases."""
    from activation_sparse_gated_gb300 import operators
    assert operators._calls is not None
    g, T, E, k, D, H = gen(91), 30, 6, 2, 128, 72
    big = torch.randn(T, 2 * D, generator=g, device=DEV).to(BF)
    x = big[:, 8:8 + D]
    W1, W3, W2t = (torch.randn(E, H, D, generator=g, device=DEV).to(BF) for _ in range(3))
    z = torch.randn(T, 2 * E, generator=g, device=DEV)[:, :E]
    q, sx = int8_operands(g, T, D)
    wq, sw = int8_operands(g, E * H, D)

    def calls():
        r = sffn.route(z, k, score="sigmoid", normalize=False)
        y = [*r, *sffn.quantize_tokens(x), sffn.matmul_int8(q, sx, wq, sw), sffn.matmul_int8(q, sx, wq, sw, dtype="f32")]
        y += [sffn.grouped_matmul(x, W1, r.offsets, index=r.rows, index_div=k),
              sffn.grouped_matmul(x[:0], W1, offsets_of([0] * E), dtype=torch.float32),
              sffn.grouped_matmul(q, wq.view(E, H, D), r.offsets, sx=sx, sw=sw.view(E, H), index=r.rows, index_div=k),
              sffn.grouped_matmul(x[:, :H], W2t, offsets_of([5] * E), transposed=1),
              sffn.experts_forward(x, r, W1, W3, W2t, act="silu")]
        return y

    one = calls()
    monkeypatch.setattr(operators, "_calls", None)
    two = calls()
    assert len(one) == len(two)
    for a, b in zip(one, two):
        assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b)
    monkeypatch.undo()
    with pytest.raises((ValueError, sffn.SffnError)):
        sffn.route(z, 10 ** 30)
    with torch.no_grad():
        w = torch.nn.Parameter(W1.clone())
        assert torch.equal(sffn.grouped_matmul(x, w, offsets_of([5] * E)), sffn.grouped_matmul(x, W1, offsets_of([5] * E)))


def test_wrappers_refuse_on_the_gpu():
    x, w = torch.zeros(4, 64, dtype=BF, device=DEV), torch.zeros(2, 8, 64, dtype=BF, device=DEV)
    off = offsets_of([2, 2])
    with pytest.raises(ValueError, match="offsets"):
        sffn.grouped_matmul(x, w, off[:2])
    with pytest.raises(ValueError, match="gradient"):
        sffn.grouped_matmul(x.clone().requires_grad_(), w, off)
    with pytest.raises(ValueError, match="contiguous"):
        sffn.grouped_matmul(x, w.transpose(0, 1), off[:1].repeat(9))
    with pytest.raises(ValueError, match="contiguous"):
        sffn.quantize_tokens(x.T)
    with pytest.raises(ValueError, match="routing"):
        sffn.experts_forward(x, sffn.route(torch.zeros(3, 2, device=DEV), 1), w, w, w)
    with pytest.raises(sffn.SffnError, match="K=60"):
        sffn.grouped_matmul(x[:, :60], w[:, :, :60].contiguous(), off)
    with pytest.raises(sffn.SffnError, match="overlap"):
        sffn.grouped_matmul(x, w, off, out=x[:, :8])


# ------------------------------------------------------------------ values that are no numbers, and values at the types' ends


# one token; few tokens (staged, too long to stage); products of one block, with K cut over a cluster, of pairs of blocks
FORMS = [(1, 8, 2, 128, 100), (5, 16, 4, 384, 130), (3, 4, 2, 6000, 24), (33, 8, 2, 520, 200), (64, 4, 2, 2560, 130),
         (4000, 8, 2, 264, 600)]


@pytest.mark.parametrize("T,E,k,D,H", FORMS)
@pytest.mark.parametrize("act", ["relu", "rsp", "silu"])
def test_experts_nan_stays_visible_and_with_its_token(T, E, k, D, H, act):
    """A token that holds a NaN comes out as NaN, however many tokens there are, and leaves the others as they are."""
    g = gen(T + D)
    x = torch.randn(T, D, generator=g, device=DEV).to(BF)
    W1, W3, W2t = ((torch.randn(E, H, D, generator=g, device=DEV) * 0.05).to(BF) for _ in range(3))
    routing = sffn.route(torch.randn(T, E, generator=g, device=DEV), k)
    clean = sffn.experts_forward(x, routing, W1, W3, W2t, act=act)
    at = T // 2
    x[at, D // 3] = math.nan
    y = sffn.experts_forward(x, routing, W1, W3, W2t, act=act)
    assert torch.isnan(y[at]).all()
    keep = [t for t in range(T) if t != at]
    assert torch.isfinite(clean).all() and torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("T,E,k,D,H", FORMS)
@pytest.mark.parametrize("act", ["relu", "rsp", "silu"])
def test_experts_dead_unit_adds_nothing(T, E, k, D, H, act):
    """A unit whose gate is 0 adds exactly 0, also where its up value overflows to infinity."""
    g = gen(T + H)
    x = (torch.rand(T, D, generator=g, device=DEV) + 0.5).to(BF)
    W1, W3, W2t = ((torch.randn(E, H, D, generator=g, device=DEV) * 0.05).to(BF) for _ in range(3))
    W1[:, 3] = -1000.0  # SiLU of less than -100 is 0 in fp32
    W3[:, 3] = 0
    routing = sffn.route(torch.randn(T, E, generator=g, device=DEV), k)
    clean = sffn.experts_forward(x, routing, W1, W3, W2t, act=act)
    W3[:, 3] = 3e38
    assert torch.equal(sffn.experts_forward(x, routing, W1, W3, W2t, act=act), clean)
    assert torch.isfinite(clean).all()


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=str)
@pytest.mark.parametrize("T,E,k", [(1, 8, 8), (5, 48, 6), (700, 48, 6), (300, 300, 8)])
def test_route_normalised_sigmoid_of_very_negative_logits(T, E, k, dtype):
    """The ratio of two sigmoids is an ordinary number where both are too small for fp32."""
    z = -85 - 115 * torch.rand(T, E, generator=gen(T + E), device=DEV)
    z[0] = -90.0
    if T > 3:
        z[1] = -86 - 3 * torch.rand(E, generator=gen(1), device=DEV)  # sigmoids at fp32's smallest normal number
        z[2] -= 3e4
        z[3] = -math.inf
        z[3, 4] = -1e30
        z[4] *= 3.4
    z = z.to(dtype)
    w, ids, _, _ = sffn.route(z, k, score="sigmoid", normalize=True)
    v = torch.sort(-z.double().cpu(), dim=1, stable=True).values[:, :k].neg()
    ls = torch.nn.functional.logsigmoid(v)
    ref = torch.exp(ls - torch.logsumexp(ls, 1, keepdim=True))
    ref[v[:, 0] < -745] = 0  # sigmoids that binary64 does not hold either: as good as masked
    # the difference of two logits is rounded once, which exp turns into that share of its result (below 1e-37 past a
    # difference of 88); exp itself 2 steps each, and a product, a quotient and sums of k terms
    tol = 88 * 2.0 ** -24 + (k + 16) * 2.0 ** -23
    torch.testing.assert_close(w.double().cpu(), ref, rtol=tol, atol=1e-37)
    assert ids[0].tolist() == list(range(k))


def largest_partial_sum(xq, wq):
    """The largest magnitude that a sum of consecutive products can have: at most twice the largest prefix's."""
    most = 0
    for row in xq:
        most = max(most, (row.long() * wq.long()).cumsum(1).abs().max().item())
    return 2 * most


@pytest.mark.parametrize("T,N,K", [(3, 90, 65536), (4, 300, 14336), (5, 90, 65536), (40, 90, 65536), (130, 200, 14336),
                                   (300, 130, 4096)])
def test_matmul_int8_is_exact_below_2_24(T, N, K):
    """Every partial sum is an integer below 2^24, so nothing but the scales is rounded, however long the sum."""
    g = gen(T + K)
    xq, sx = int8_operands(g, T, K)
    wq, sw = int8_operands(g, N, K)
    assert largest_partial_sum(xq, wq) < 2 ** 24
    ref = (xq.double() @ wq.double().T) * torch.outer(sx.double(), sw.double())
    close(sffn.matmul_int8(xq, sx, wq, sw, dtype="f32"), ref, 2 * 2.0 ** -24 * ref.abs())
    off = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    y = sffn.grouped_matmul(xq, wq.expand(2, N, K).contiguous(), off, sx=sx, sw=sw.expand(2, N).contiguous(), dtype="f32")
    close(y, ref, 2 * 2.0 ** -24 * ref.abs())


@pytest.mark.parametrize("T,N,K", [(1, 64, 65536), (4, 64, 2048), (4, 64, 14336), (4, 64, 65536), (5, 64, 2048),
                                   (5, 64, 14336), (5, 64, 65536), (130, 200, 14336), (300, 130, 65536),
                                   (2048, 2048, 4096), (2100, 3001, 14336)])
def test_matmul_int8_sums_past_2_24(T, N, K):
    """Codes of one sign, so that every sum passes 2^24.  Up to four rows sum in int32 and round once; the tensor cores
    add 16 products and the running sum at a time in fp32, each of the 17 terms cut to the last place of the largest.
    The running sum grows evenly, so n = K / 16 steps lose less than 17 * 2^-23 * (n + 1) / 2 of the sum, and blocks that
    share K join at most eight parts."""
    g = gen(T + K)
    xq = torch.randint(100, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    wq = torch.randint(100, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    sx, sw = (torch.rand(n, generator=g, device=DEV) + 0.5 for n in (T, N))
    total = xq.double() @ wq.double().T
    assert total.min() > 2 ** 24
    ref = total * torch.outer(sx.double(), sw.double())
    share = 2.0 ** -24 if T <= 4 else 17 * 2.0 ** -23 * (K / 16 + 1) / 2 + 8 * 2.0 ** -23
    close(sffn.matmul_int8(xq, sx, wq, sw, dtype="f32"), ref, (share * 1.01 + 3 * 2.0 ** -24) * ref)


def test_quantize_as_many_tokens_as_an_int_counts():
    """The last tokens' numbers are within a step of 2^31: a block's next token must not turn negative."""
    T = 2 ** 31 - 100
    x = torch.ones(T, 1, device=DEV, dtype=BF)
    x[-3:, 0] = torch.tensor([0.0, -254.0, 2.0], dtype=BF, device=DEV)
    q, s = sffn.quantize_tokens(x)
    assert s[-3:].tolist() == [0.0, 2.0, torch.tensor(2.0).div(127).item()] and q[-3:, 0].tolist() == [0, -127, 127]
    assert (q[:-3] == 127).all() and (s[:-3] == torch.tensor(1.0, device=DEV).div(127)).all()


@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_moe_keeps_a_corrupted_token_visible(T, bad):
    g, E, D, H = gen(T), 6, 128, 200
    x = torch.randn(T, D, generator=g, device=DEV).to(BF)
    Wr = torch.randn(E, D, generator=g, device=DEV)
    W1, W3, W2 = (torch.randn(E, a, b, generator=g, device=DEV).to(BF) for a, b in ((H, D), (H, D), (D, H)))
    moe = sffn.MoEFFN(Wr, W1, W3, W2, 2)
    clean = moe(x)
    x[T // 2, 7] = bad
    y = moe(x)
    assert not torch.isfinite(y[T // 2]).any()
    keep = [t for t in range(T) if t != T // 2]
    assert torch.equal(y[keep], clean[keep]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("tf32", [False, True])
@pytest.mark.parametrize("T", [1, 7, 300])
def test_moe_choice_does_not_follow_the_tf32_switch(T, tf32):
    """Experts whose logits differ by less than TF32 resolves are told apart, whatever the process-wide switch says."""
    g, E, D, H = gen(T), 4, 256, 64
    x = (torch.rand(T, D, generator=g, device=DEV) + 0.5).to(BF)
    Wr = (1 + torch.arange(E, device=DEV) * 2.0 ** -13)[:, None].expand(E, D).contiguous()  # TF32 steps by 2^-10
    W1, W3 = (torch.randn(E, H, D, generator=g, device=DEV).to(BF) for _ in range(2))
    # an fp32 logit is off by D steps of 2^-23 at most, 2^-15 of its sum: a quarter of the gaps
    moe = sffn.MoEFFN(Wr, W1, W3, W3.transpose(1, 2), 2)
    before = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = tf32
    try:
        ids = moe.route(x).ids
    finally:
        torch.backends.cuda.matmul.allow_tf32 = before
    assert ids.tolist() == [[E - 1, E - 2]] * T


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, BF], ids=str)
@pytest.mark.parametrize("T,E,D", [(0, 5, 64), (1, 64, 2560), (9, 7, 72), (400, 100, 1032)])
def test_moe_router_product(T, E, D, dtype):
    """The layer's weights against the softmax in 64 bits of all of Wr's bits."""
    g = gen(T + D)
    x = torch.randn(T, 2 * D, generator=g, device=DEV).to(BF)[:, 8:8 + D]
    Wr = (torch.randn(E, D, generator=g, device=DEV) * 0.1).to(dtype)
    W = torch.zeros(E, 8, D, device=DEV, dtype=BF)
    weights, ids, _, _ = sffn.MoEFFN(Wr, W, W, W.transpose(1, 2), E if E < 32 else 32, normalize=False).route(x)
    z, mag = x.double() @ Wr.double().T, x.double().abs() @ Wr.double().abs().T
    # D steps of the product and three of the parts' sum, on logits; exp turns twice the largest into a share, and adds
    # two steps of its own and those of a sum of E terms and a quotient
    dz = (D + 4) * 2.0 ** -23 * mag.amax(1, keepdim=True)
    p = torch.softmax(z, 1)
    picked = p.gather(1, ids.long())
    tol = picked * (2.1 * dz + (E + 8) * 2.0 ** -23)
    assert ((weights.double() - picked).abs() <= tol).all()
    # the chosen are the largest, as far as the logits' bounds tell them apart
    left = z.scatter(1, ids.long(), -math.inf).amax(1, keepdim=True)
    assert (z.gather(1, ids.long()) + 2 * dz >= left).all()


def dual_calls():
    import torch.autograd.forward_ad as fw
    g, E, k, D, H = gen(95), 4, 2, 64, 32
    x = torch.randn(6, D, generator=g, device=DEV).to(BF)
    W1, W3, W2t = (torch.randn(E, H, D, generator=g, device=DEV).to(BF) for _ in range(3))
    z = torch.randn(6, E, generator=g, device=DEV)
    q, sx = int8_operands(g, 6, D)
    wq, sw = int8_operands(g, H, D)
    r, off = sffn.route(z, k), offsets_of([2, 0, 1, 3])
    dual = lambda t: fw.make_dual(t, torch.ones_like(t))  # noqa: E731
    return {"route": lambda: sffn.route(dual(z), k),
            "quantize": lambda: sffn.quantize_tokens(dual(x)),
            "int8 sx": lambda: sffn.matmul_int8(q, dual(sx), wq, sw),
            "int8 sw": lambda: sffn.matmul_int8(q, sx, wq, dual(sw)),
            "grouped x": lambda: sffn.grouped_matmul(dual(x), W1, off),
            "grouped w": lambda: sffn.grouped_matmul(x, dual(W1), off),
            "experts x": lambda: sffn.experts_forward(dual(x), r, W1, W3, W2t),
            "experts weights": lambda: sffn.experts_forward(x, (dual(r.weights), *r[1:]), W1, W3, W2t),
            "experts W2t": lambda: sffn.experts_forward(x, r, W1, W3, dual(W2t))}


@pytest.mark.parametrize("which", ["route", "quantize", "int8 sx", "int8 sw", "grouped x", "grouped w", "experts x",
                                   "experts weights", "experts W2t"])
def test_forward_mode_tangents_are_refused(which):
    import torch.autograd.forward_ad as fw
    with fw.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            dual_calls()[which]()
