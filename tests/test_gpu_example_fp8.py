"""The example that trains a linear layer with FP8 products: it runs, its gradients are those of the quantized layer, and
its updates use the clipped ones."""
import importlib.util
import math
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import f8_ref as ref


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_step.py")
    spec = importlib.util.spec_from_file_location("fp8_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("sizes", [dict(tokens=1, k=8, n=8), dict(tokens=130, k=264, n=136), {}], ids=str)
def test_it_runs(example, sizes):
    layer, losses = example.train(steps=3, say=lambda *_: None, **sizes)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
    assert torch.isfinite(layer.master).all() and torch.isfinite(layer.dw).all()


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def values(t, direction, fmt, use_2d=False):
    q = ref.quantize(bits(t), direction, fmt, use_2d)
    return ref.values(*q, fmt)[0]


def test_gradients_and_update(example):
    """y, dx and dw against 64-bit products of the quantized operands.  A product's error is below 2^-9 of the sum of its
    magnitudes (each product loses at most 2^-13 of the largest of its 8, so a group of 8 loses 7 2^-13 of its own sum of
    magnitudes at most, and fp32 sums of 300 terms 300 2^-24); bf16 rounds by 2^-8 more."""
    layer = example.Linear(264, 136, max_norm=1e-2, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(300, 264, device="cuda", generator=gen).bfloat16()
    dy = (torch.randn(300, 136, device="cuda", generator=gen) * 1e-2).bfloat16()
    layer.b16.fill_(0.5)
    y = layer.forward(x)
    dx = layer.backward(dy)

    def check(got, a, b, rounds, add=0.0):
        want, size = a @ b.T + add, np.abs(a) @ np.abs(b).T
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= 2.0 ** -9 * size + rounds * (np.abs(want) + 2.0 ** -9 * size)).all()

    check(y, values(x, 0, 0)[:, :264], values(layer.w, 0, 0, True)[:, :264], 2.0 ** -8, 0.5)
    check(dx, values(dy, 0, 1)[:, :136], values(layer.w, 1, 0, True)[:, :136], 2.0 ** -8)
    check(layer.dw, values(dy, 1, 1)[:, :300], values(x, 1, 0)[:, :300], 0.0)
    total = math.sqrt(layer.dw.double().square().sum().item() + layer.db.double().square().sum().item())
    assert total > 1e-2
    layer.update(1, 1e-3)
    assert abs(layer.norm().item() - total) <= 2.0 ** -22 * total
    # AdamW's first moment of the first step: 0.1 of the clipped gradient
    m = layer.states[0][0].double()
    want = 0.1 * layer.dw.double() * (1e-2 / (total + 1e-6))
    assert (m - want).abs().max() <= 2.0 ** -21 * want.abs().max()
