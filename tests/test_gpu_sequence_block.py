"""examples/sequence_block.py: the operators together.  It learns its task with
32-bit and with 8-bit moments, and answering token by token gives the logits of
the whole-sequence pass."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("sequence_block", os.path.join(ROOT, "examples", "sequence_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_learns(example, bits):
    """16 symbols: a guess costs log 16 = 2.77; the delayed copy is within the convolution's reach, so the
    loss must fall below a quarter of that."""
    model, losses = example.train(steps=150, bits=bits)
    assert abs(losses[0] - 2.77) < 1.0 and losses[-1] < 0.69, (losses[0], losses[-1])


def test_token_by_token_equals_whole_sequence(example):
    model, _ = example.train(steps=5)
    ids, _, _ = example.batch(torch.Generator(device="cuda").manual_seed(7), 3, 80, model.symbols)
    whole, _ = model.forward(ids)
    state = model.start(3)
    steps = torch.stack([model.answer(ids[:, t], state) for t in range(80)], 1)
    # the recurrence's two forms round differently, and each value passes two bf16 roundings after it
    scale = whole.abs().amax()
    assert float((steps - whole).abs().amax()) <= 4 * 2.0 ** -8 * float(scale)
