"""The example that trains a layer of experts: its loss falls, and small and ragged layers run."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "experts_step.py")
    spec = importlib.util.spec_from_file_location("experts_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_layer_of_experts_learns(example):
    """The target has unit output variance, so the loss starts near 1.  What quantization leaves: x and w carry a
    relative error of at most about 0.15 each in the mean square root (half steps of E2M1 under a shared scale), a
    floor of 2 * 0.15^2 = 0.045 once w fits; half of the start is far above it."""
    losses = example.train(steps=60, tokens=512, experts=8, topk=2, k=256, n=128, say=lambda *_: None)
    assert 0.7 < losses[0] < 1.4
    assert losses[-1] < 0.5 * losses[0]
    assert all(v == v for v in losses)


@pytest.mark.parametrize("sizes", [dict(tokens=1, experts=3, topk=1, k=8, n=8), dict(tokens=37, experts=5, topk=3, k=72, n=40)])
def test_small_layers_run(example, sizes):
    assert len(example.train(steps=3, say=lambda *_: None, **sizes)) == 3
