"""The example of a KDA layer and a layer of latent attention, prompts against
single tokens."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,steps,heads", [(300, 4, 4), (70, 1, 2), (3, 2, 8)])
def test_steps_continue_a_prompt(example, tokens, steps, heads):
    # Both ways round the same values to 8 bits (e4m3: 2^-4 of a value); they differ where a bf16 rounding before
    # (2^-8) moves a value over an 8-bit boundary: at most one half step on average.
    assert example.compare(tokens, steps, heads) < 2.0 ** -4
