"""The example of a KDA layer and a layer of latent attention with rotary positions
and the quantised cache: prompts, prompts behind prompts, single tokens."""
import pytest
import torch

from test_gpu_hybrid_layers import example  # noqa: F401

pytestmark = pytest.mark.gpu


def inputs(counts, more, dim=1024, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda n: torch.randn(n, dim, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    return [new(c) for c in counts], [new(m) for m in more]


# Both ways round the same values to 8 bits (e4m3: 2^-4 of a value); they differ where a bf16 rounding before (2^-8) moves a
# value over an 8-bit boundary: at most one half step on average, in the projections and in the cache.
ROOM = 2 * 2.0 ** -4


@pytest.mark.parametrize("tokens,steps,heads", [(300, 4, 4), (70, 1, 2), (3, 2, 8)])
def test_steps_continue_a_prompt(example, tokens, steps, heads):  # noqa: F811
    assert example.compare(tokens, steps, heads, quantized=True) < ROOM


@pytest.mark.parametrize("counts,more,heads", [([200, 65, 1], [100, 3, 130], 4), ([64, 1, 30], [1, 64, 500], 2)])
def test_prompts_go_on_behind_cached_prompts(example, counts, more, heads):  # noqa: F811
    """In two parts, the second over what is read back of the first, and as one: the last hidden states, and the cache."""
    first, second = inputs(counts, more)
    both = [a + b for a, b in zip(counts, more)]
    model = example.Stack(1024, heads, 0, quantized=True)
    model.prompt(torch.cat(first), counts, max(both))
    split = model.more(torch.cat(second), more)
    layer = model.latent
    assert layer.lens.tolist() == both

    def cached():
        kda = example.kda
        cu = torch.tensor([0] + both).cumsum(0).to("cuda", torch.int32)
        c, r = kda.latent_cache_read(layer.cache, layer.table, layer.lens, cu, total_tokens=sum(both), page_size=example.PAGE, dtype=torch.float32)
        return torch.cat([c, r], 1)
    parts = cached()
    whole = model.prompt(torch.cat([torch.cat([a, b]) for a, b in zip(first, second)]), both, max(both))
    last = whole[torch.tensor(both, device="cuda").cumsum(0) - 1].float()
    got = split[torch.tensor(more, device="cuda").cumsum(0) - 1].float()
    off = (got - last).norm(dim=1) / last.norm(dim=1)
    assert float(off.max()) < 2 * ROOM, off
    one = cached()
    off = (parts - one).norm(dim=1) / one.norm(dim=1)
    assert float(off.max()) < 2 * ROOM, off.topk(4)
