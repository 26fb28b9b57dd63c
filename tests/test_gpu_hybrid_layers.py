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


@pytest.mark.parametrize("tokens,steps,heads", [(300, 4, 4), (70, 3, 2)])
def test_steps_leave_the_cache_of_one_longer_prompt(example, tokens, steps, heads):
    """Token by token: a latent of another token, or none, is off by about its own size.  Between the two ways lie two
    8-bit roundings in a row (the norm's output, and the mixer's behind it), of 2^-4 of a value each."""
    counts, dim = [tokens, tokens // 3, 1], 1024
    g = torch.Generator(device="cuda").manual_seed(5)
    new = lambda n: torch.randn(n, dim, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    prompts, more = [new(c) for c in counts], [new(len(counts)) for _ in range(steps)]
    model = example.Stack(dim, heads, 0)
    longer = [c + steps for c in counts]

    def cached():
        layer = model.latent
        assert layer.lens.tolist() == longer
        rows = layer.cache[layer.table.long()].flatten(1, 2)
        return torch.cat([rows[i, :n] for i, n in enumerate(longer)]).float()
    model.prompt(torch.cat(prompts), counts, max(longer))
    for x in more:
        model.step(x)
    stepped = cached()
    model.prompt(torch.cat([torch.cat([p] + [x[i:i + 1] for x in more]) for i, p in enumerate(prompts)]), longer, max(longer))
    whole = cached()
    off = (stepped - whole).norm(dim=1) / whole.norm(dim=1)
    assert float(off.max()) < 2 * 2.0 ** -4, off.topk(4)
