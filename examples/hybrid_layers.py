"""Two layers of a hybrid stack served with the package's calls: a KDA layer and a
layer of latent attention, prompts first, then one token at a time.

    python examples/hybrid_layers.py [--tokens 300] [--steps 4] [--heads 4]

Each layer is: norm of the residual stream with an 8-bit output (rms_norm),
8-bit projections (matmul_fp8), its mixer (prefill / decode_step, or
latent_prefill / latent_decode over a paged cache), a norm of the mixer's output
and an 8-bit output projection.  Weights are random.  The script feeds a prompt,
continues it token by token, feeds prompt and continuation again as one prompt,
and prints how far the two last hidden states are apart.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_gated_delta_chunked_gb300 as kda  # noqa: E402

D_HEAD, RANK, ROPE, PAGE = 128, 512, 64, 64


class Linear8:
    """A weight [n, k] in e4m3 with one scale for each 128 x 128 block."""

    def __init__(self, n: int, k: int, g: torch.Generator):
        w = torch.randn(n, k, generator=g, device="cuda") / k ** 0.5
        nb, kb = -(-n // 128), -(-k // 128)
        blocks = torch.nn.functional.pad(w, (0, kb * 128 - k, 0, nb * 128 - n)).view(nb, 128, kb, 128)
        self.scale = (blocks.abs().amax((1, 3)) / 448).contiguous()
        q = (blocks / self.scale[:, None, :, None]).reshape(nb * 128, kb * 128)[:n, :k]
        self.weight = q.to(torch.float8_e4m3fn).contiguous()

    def __call__(self, x8, x_scale):
        return kda.matmul_fp8(x8, x_scale, self.weight, self.scale)

    def dense(self) -> torch.Tensor:
        n, k = self.weight.shape
        s = self.scale.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        return (self.weight.float() * s).to(torch.bfloat16)


class KdaLayer:
    def __init__(self, dim: int, heads: int, g: torch.Generator):
        self.heads, width = heads, heads * D_HEAD
        self.norm = torch.ones(dim, device="cuda", dtype=torch.bfloat16)
        self.qkv, self.gates = Linear8(3 * width, dim, g), Linear8(width + heads, dim, g)
        self.out = Linear8(dim, width, g)
        self.state = None

    def _inputs(self, x8, xs):
        t, h = x8.shape[0], self.heads
        q, k, v = (y.view(t, h, D_HEAD) for y in self.qkv(x8, xs).split(h * D_HEAD, 1))
        gate = self.gates(x8, xs).float()
        unit = lambda y: torch.nn.functional.normalize(y.float(), dim=-1)  # noqa: E731
        log_alpha = -0.1 * torch.sigmoid(gate[:, :h * D_HEAD]).view(t, h, D_HEAD)
        beta = torch.sigmoid(gate[:, h * D_HEAD:])
        return [y.to(torch.bfloat16).contiguous() for y in (unit(q) / D_HEAD ** 0.5, unit(k), v, log_alpha, beta)]

    def __call__(self, x, residual, lengths):
        """One packed prompt a sequence (lengths given), or one token a sequence (None)."""
        _, x8, xs, residual = kda.rms_norm(x, self.norm, residual, normed=False, quantize=True)
        y = self._inputs(x8, xs)
        if lengths is None:
            o = kda.decode_step(*y, self.state)
        else:
            o, self.state, _ = kda.prefill(*y, lengths)
        _, o8, os_, _ = kda.rms_norm(o.view(x.shape[0], -1), normed=False, quantize=True)
        return self.out(o8, os_), residual


class LatentLayer:
    def __init__(self, dim: int, heads: int, g: torch.Generator):
        self.heads, self.scale = heads, (D_HEAD + ROPE) ** -0.5
        self.norm = torch.ones(dim, device="cuda", dtype=torch.bfloat16)
        self.latent_norm = torch.ones(RANK, device="cuda", dtype=torch.bfloat16)
        self.q = Linear8(heads * (D_HEAD + ROPE), dim, g)
        self.down = Linear8(RANK + ROPE, dim, g)
        self.up = Linear8(heads * 2 * D_HEAD, RANK, g)            # a head's keys, then its values
        self.out = Linear8(dim, heads * D_HEAD, g)
        up = self.up.dense().view(heads, 2, D_HEAD, RANK)
        self.up_k, self.up_v = up[:, 0].contiguous(), up[:, 1].contiguous()

    def start(self, sequences: int, capacity: int):
        """An empty cache with room for `capacity` tokens a sequence."""
        per = -(-capacity // PAGE)
        self.cache = torch.zeros(sequences * per, PAGE, RANK + ROPE, device="cuda", dtype=torch.bfloat16)
        self.table = torch.randperm(sequences * per, device="cuda").to(torch.int32).view(sequences, per)
        self.lens = torch.zeros(sequences, device="cuda", dtype=torch.int32)

    def _append(self, latent, rope, lengths):
        """Tokens of each sequence (counts on the host) behind those in the cache."""
        seq = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths)).cuda()
        first = torch.tensor([0] + lengths).cumsum(0)[:-1].cuda()
        at = torch.arange(latent.shape[0], device="cuda") - first[seq] + self.lens[seq]
        rows = self.table[seq, at // PAGE].long() * PAGE + at % PAGE
        self.cache.view(-1, RANK + ROPE)[rows] = torch.cat([latent, rope], 1)
        self.lens += torch.tensor(lengths, device="cuda", dtype=torch.int32)

    def __call__(self, x, residual, lengths, counts):
        _, x8, xs, residual = kda.rms_norm(x, self.norm, residual, normed=False, quantize=True)
        t, h = x.shape[0], self.heads
        q = self.q(x8, xs).view(t, h, D_HEAD + ROPE)
        down = self.down(x8, xs)
        rope = down[:, RANK:]
        latent, c8, cs, _ = kda.rms_norm(down[:, :RANK], self.latent_norm, quantize=True)
        self._append(latent, rope, counts)
        if lengths is None:                                       # the up-projections folded into queries and output
            q_latent = torch.einsum("nhd,hdr->nhr", q[..., :D_HEAD], self.up_k)
            o, _ = kda.latent_decode(torch.cat([q_latent, q[..., D_HEAD:]], -1), self.cache, self.table, self.lens,
                                     scale=self.scale)
            o = torch.einsum("nhr,hdr->nhd", o, self.up_v)
        else:
            kv = self.up(c8, cs).view(t, h, 2 * D_HEAD)
            o, _ = kda.latent_prefill(q, kv[..., :D_HEAD], rope, kv[..., D_HEAD:], lengths, lengths, scale=self.scale)
        _, o8, os_, _ = kda.rms_norm(o.reshape(t, -1), normed=False, quantize=True)
        return self.out(o8, os_), residual


class Stack:
    def __init__(self, dim: int = 1024, heads: int = 4, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kda, self.latent = KdaLayer(dim, heads, g), LatentLayer(dim, heads, g)

    def prompt(self, x, counts, capacity):
        """x [sum of counts, dim]: hidden states of packed prompts.  Returns those behind the two layers."""
        self.latent.start(len(counts), capacity)
        lengths = torch.tensor([0] + counts).cumsum(0).to("cuda", torch.int32)
        return self._run(x, lengths, counts)

    def step(self, x):
        """x [sequences, dim]: the hidden state of one more token of each."""
        return self._run(x, None, [1] * x.shape[0])

    def _run(self, x, lengths, counts):
        y, residual = self.kda(x, torch.zeros_like(x), lengths)
        y, residual = self.latent(y, residual, lengths, counts)
        return y + residual


def compare(tokens: int = 300, steps: int = 4, heads: int = 4, dim: int = 1024, seed: int = 0) -> float:
    """Relative difference of the last hidden states: prompt and steps, against one longer prompt."""
    counts = [tokens, max(1, tokens // 3), 1]
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    new = lambda n: torch.randn(n, dim, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    prompts, more = [new(c) for c in counts], [new(len(counts)) for _ in range(steps)]
    model = Stack(dim, heads, seed)
    model.prompt(torch.cat(prompts), counts, max(counts) + steps)
    for x in more:
        stepped = model.step(x)
    whole = [torch.cat([p] + [x[i:i + 1] for x in more]) for i, p in enumerate(prompts)]
    longer = [c + steps for c in counts]
    full = model.prompt(torch.cat(whole), longer, max(longer))
    last = full[torch.tensor(longer, device="cuda").cumsum(0) - 1]
    return float((stepped.float() - last.float()).norm() / last.float().norm())


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=300)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--heads", type=int, default=4)
    a = p.parse_args()
    print(f"prompt + {a.steps} steps against one prompt: relative difference {compare(a.tokens, a.steps, a.heads):.2e}")
