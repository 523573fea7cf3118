"""The signs of the gates that a training step keeps, and its gradients from x and the weights on, against 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
import activation_sparse_gated_gb300 as sffn  # noqa: E402
from test_gpu_gated_int4 import BF, DEV, close, gen, grads, no_device_error, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def cancelling(g, T, D, H, jump=False):
    """x [T, D] and W [H, D] whose sums rise to hundreds and come back to a few 2^-20: the second half of a row of W is the
    first half's negative, and a last column decides the sign.  ``jump``: they do so in the first and the last columns, and
    stay up between.  Every product is a multiple of 2^-40 and every sum below 2^13, so 64 bits hold them exactly."""
    n = (D - 8) // 2

    def values(rows):
        v = 1 + torch.randint(0, 128, (rows, n), generator=g, device=DEV) / 128.0
        return v * 2.0 ** -torch.randint(0, 4, (rows, n), generator=g, device=DEV)

    a, b = values(T), values(H)
    if jump:
        b[:, 16:] *= 2.0 ** -8
    b2 = b.flip(1) if jump else b
    a2 = a.flip(1) if jump else a
    x, W = torch.zeros(T, D, device=DEV), torch.zeros(H, D, device=DEV)
    x[:, :n], x[:, n:2 * n], x[:, -1] = a, a2, 1
    W[:, :n], W[:, n:2 * n] = b, -b2
    W[:, -1] = torch.randint(-7, 8, (H,), generator=g, device=DEV) * 2.0 ** -20
    return x.to(BF), W.to(BF)


# one token and short last pieces of layers whose sums are not cut, sums cut over a cluster, tiles of a pair, narrow layers
CANCELLING = [(1, 520, 14336), (33, 520, 10001), (65, 264, 9000), (257, 2568, 300), (3, 264, 17), (17, 136, 5), (40, 136, 1),
              (700, 1032, 2000), (2048, 520, 4100)]


@pytest.mark.parametrize("T,D,H", CANCELLING)
@pytest.mark.parametrize("act,jump", [("relu", False), ("rsp", True)])
def test_the_sign_of_a_kept_gate_is_the_exact_sums(T, D, H, act, jump):
    """Every z here is within the tensor cores' error of 0.  A token's size and its neighbours' make no difference."""
    g = gen(T + D + H)
    x, W1 = cancelling(g, T, D, H, jump)
    x[T // 3] *= 2.0 ** -30
    x[T // 2] *= 2.0 ** 10
    W1[H // 3] *= 2.0 ** -12
    W1[H // 2] = 0
    W3 = randn(g, H, D)
    h, z, u = sffn.gated_up_saved(x, W1, W3, act=act)
    ref = x.double() @ W1.double().T
    wrong = (z > 0) != (ref > 0)
    assert not wrong.any(), f"{int(wrong.sum())} of {T * H} signs"
    close(z, ref, 0.0)
    if act == "relu":
        assert torch.equal(h, torch.where(z > 0, z * u, torch.zeros_like(z)).to(BF))
    else:
        assert (h[z <= 0] == 0).all()


@pytest.mark.parametrize("T,H", [(70, 9000), (70, 200)])
def test_signs_beside_tokens_that_are_no_numbers(T, H):
    g = gen(5)
    x, W1 = cancelling(g, T, 520, H)
    W3 = randn(g, H, 520)
    x[3, 7], x[35, 100], x[36, 2] = math.nan, math.inf, -math.inf
    x[50] = 0
    _, z, _ = sffn.gated_up_saved(x, W1, W3, act="relu")
    assert torch.isnan(z[3]).all() and not torch.isfinite(z[35:37]).any() and (z[50] == 0).all()
    keep = torch.tensor([t not in (3, 35, 36) for t in range(T)], device=DEV)
    assert torch.equal(z[keep] > 0, x[keep].double() @ W1.double().T > 0)


@pytest.mark.parametrize("of_x,of_W", [(2.0 ** -50, 2.0 ** -50), (2.0 ** 58, 2.0 ** -50), (2.0 ** -50, 2.0 ** 58)])
def test_signs_of_small_and_large_values(of_x, of_W):
    """Squares of these leave fp32, their products do not."""
    g = gen(6)
    x, W1 = cancelling(g, 50, 520, 300)
    x, W1 = x * of_x, W1 * of_W
    _, z, _ = sffn.gated_up_saved(x, W1, randn(g, 300, 520), act="relu")
    ref = x.double() @ W1.double().T
    assert torch.equal(z > 0, ref > 0)
    close(z, ref, 0.0)


@pytest.mark.parametrize("T,D,H", [(1, 64, 33), (5, 328, 9), (60, 2560, 500), (1000, 640, 1024), (1500, 2560, 2600)])
@pytest.mark.parametrize("act", ["relu", "rsp", "silu"])
def test_gradients_from_the_inputs_on(T, D, H, act):
    """A step by autograd against the formula from x, W1 and W3.  x, W1 and W3 are multiples of 2^-3 and 2^-6 and sums stay
    below 2^10, so that every sum is exact in fp32 in any order, and every sign is defined."""
    g = gen(T + D)

    def grid(rows, most, step):
        return (torch.randint(-most, most + 1, (rows, D), generator=g, device=DEV) * step).to(BF)

    x, W1, W3 = grid(T, 8, 2.0 ** -3), grid(H, 16, 2.0 ** -6), grid(H, 16, 2.0 ** -6)
    x[:, -1], W1[:, -1] = 1, -1.25
    dh = randn(g, T, H)
    leaves = [t.clone().requires_grad_() for t in (x, W1, W3)]
    sffn.gated_up(*leaves, act=act).backward(dh)
    z, u = x.double() @ W1.double().T, x.double() @ W3.double().T
    for t, (ref, bound) in zip(leaves, grads(dh, z, u, x, W1, W3, act)):
        close(t.grad, ref, bound)


def test_a_step_of_gates_next_to_0_by_its_gradients():
    """The same for sums that the tensor cores would get wrong."""
    g = gen(8)
    T, D, H = 300, 1032, 640
    x, W1 = cancelling(g, T, D, H)
    W1[:H // 2] = randn(g, H // 2, D) * D ** -0.5  # half of the units are ordinary
    W3, dh = randn(g, H, D) * D ** -0.5, randn(g, T, H)
    leaves = [t.clone().requires_grad_() for t in (x, W1, W3)]
    for act in ("relu", "rsp"):
        for t in leaves:
            t.grad = None
        sffn.gated_up(*leaves, act=act).backward(dh)
        z, u = x.double() @ W1.double().T, x.double() @ W3.double().T
        S = x.double().abs() @ W3.double().abs().T
        du = (D + 8) * 2.0 ** -23 * S  # u and the ordinary units' z are sums of the tensor cores'
        dzo = 1.1 * dh.double().abs() * du
        Z = (D + 8) * 2.0 ** -23 * (x.double().abs() @ W1.double().abs().T)
        duo = dh.double().abs() * 1.1 * Z
        dzo = dzo + duo * u.abs()
        more = (dzo @ W1.double().abs() + duo @ W3.double().abs(), dzo.T @ x.double().abs(), duo.T @ x.double().abs())
        for t, (ref, bound), m in zip(leaves, grads(dh, z, u, x, W1, W3, act), more):
            close(t.grad, ref, bound + 1.01 * m)


def test_signs_in_a_captured_step_and_on_two_streams():
    """The norms that the signs go by wait in the results' memory: nothing of them is left, and calls do not meet."""
    g = gen(9)
    x, W1 = cancelling(g, 130, 520, 9000)
    W3 = randn(g, 9000, 520)
    want = sffn.gated_up_saved(x, W1, W3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sffn.gated_up_saved(x, W1, W3)
    for _ in range(3):
        for t in got:
            t.fill_(math.nan)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    many = [sffn.gated_up_saved(x, W1, W3, stream=s) for _ in range(6) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in many for a, b in zip(r, want))


@pytest.mark.parametrize("T,H", [(1, 9000), (50, 9001), (50, 77), (600, 2100)])
def test_results_with_pitches_of_their_own(T, H):
    """z, u and h in rows that are longer than they are and start anywhere: what lies between stays."""
    g = gen(11)
    D, ld = 520, H + 37
    x, W1 = cancelling(g, T, D, H)
    W3 = randn(g, H, D)
    h, z, u = (torch.full((T, ld), 5.0, dtype=t, device=DEV) for t in (BF, torch.float32, torch.float32))
    rc = sffn.load().sffn_gated_up(x.data_ptr(), D, W1.data_ptr(), W3.data_ptr(), h.data_ptr() + 2 * 3, ld, z.data_ptr() + 4 * 5,
                                   u.data_ptr() + 4 * 7, ld, T, D, H, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == sffn.SFFN_OK
    want = sffn.gated_up_saved(x, W1, W3)
    for t, first, w in ((h, 3, want[0]), (z, 5, want[1]), (u, 7, want[2])):
        assert torch.equal(t[:, first:first + H], w)
        assert (t[:, :first] == 5).all() and (t[:, first + H:] == 5).all()
