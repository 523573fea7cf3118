"""The gated block and the 4-bit products in the forms that the launch rules give to real layers, and their refusals."""
import pytest

torch = pytest.importorskip("torch")
import activation_sparse_gated_gb300 as sffn  # noqa: E402
from test_gpu_gated_int4 import BF, DEV, gen, no_device_error, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,H", [(2, 65544, 4), (2, 64, 65537)])
def test_sizes_past_the_limit_raise_the_same_error_with_and_without_gradients(T, D, H):
    g = gen(1)
    x, W1, W3 = randn(g, T, D), randn(g, H, D), randn(g, H, D)
    for leaf in (None, x, W1, W3):
        args = [t.clone().requires_grad_() if t is leaf else t for t in (x, W1, W3)]
        with pytest.raises(sffn.SffnError, match="at most"):
            sffn.gated_up(*args)
