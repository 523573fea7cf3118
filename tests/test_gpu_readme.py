"""The README's Python examples run as they stand, on tensors of the kinds that their comments say."""
import os
import re

import pytest

torch = pytest.importorskip("torch")
import activation_sparse_gated_gb300 as sffn  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def examples():
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        return re.findall(r"```python\n(.*?)```", f.read(), re.S)


def names(T=24, D=64, H=128, E=8, grad=False):
    g = torch.Generator(device="cuda").manual_seed(1)

    def t(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    many = () if grad else (E,)
    one = {"x": t(T, D), "W1": t(*many, H, D), "W3": t(*many, H, D), "W2": t(*many, D, H)}
    if grad:
        for v in one.values():
            v.requires_grad_()
        return {**one, "torch": torch, "sffn": sffn, "dy": t(T, D), "dh": t(T, H), "W": t(H, D)}
    wq, sw = sffn.quantize_tokens(t(H, D))
    return {**one, "Wr": t(E, D), "W2t": one["W2"].transpose(1, 2).contiguous(), "logits": t(T, E), "wq": wq, "sw": sw}


def test_every_example_is_run(cuda_ok):
    found = examples()
    assert len(found) == 2
    for text in found:
        exec(text, names(grad="gated_up" in text))  # noqa: S102
    sffn.sffn_check()
