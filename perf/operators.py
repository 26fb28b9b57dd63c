"""Cases, plain forms and 64-bit definitions of the operators around a KDA stack's global layer.

A KDA model alternates its recurrent layers with layers of full attention whose
keys and values come from one shared latent vector a token, and the projections
of both run in 8-bit floating point behind a root-mean-square norm.  Four calls:

  norm     h = x + r;  y = h / sqrt(mean(h^2) + eps) * w, given as y and/or as
           e4m3 values with one fp32 scale for each 128 of a row
  matmul   C[m, n] = sum_k A[m, k] sa[m, k/128] B[n, k] sb[n/128, k/128], A and B e4m3
  expanded causal attention of packed prompts, keys [k_nope | k_rope] (k_rope
           shared by the heads), values of their own
  absorbed attention of one or a few tokens a sequence over a paged cache of
           latents c = [c_value | c_rope]; keys are c, values its first 512

``own`` selects between the plain form (elementary torch operations in 32 bits)
and the package's calls.
"""
import math

import torch

own = False

RANK, ROPE, NOPE, VDIM = 512, 64, 128, 128
DEV = "cuda"


def listed():
    return [
        # one decoded token: the norm before a projection, latency alone
        {"name": "norm_token", "op": "norm", "tokens": 1, "dim": 4096, "dtype": "bf16", "residual": True, "normed": False, "quant": True},
        # an odd batch with rows that no vector width divides, plain normed output, 32-bit activations
        {"name": "norm_odd_f32", "op": "norm", "tokens": 777, "dim": 2051, "dtype": "f32", "residual": True, "normed": True, "quant": False},
        # a long prompt's activations, both outputs (the gates read the 16-bit one, the projections the 8-bit one)
        {"name": "norm_prompt", "op": "norm", "tokens": 65536, "dim": 4096, "dtype": "bf16", "residual": True, "normed": True, "quant": True},
        # one decoded token through a square projection: the weights' bytes
        {"name": "matmul_token", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "out": "bf16"},
        # a decode batch of 256 sequences through the query projection of 32 heads x 192
        {"name": "matmul_batch", "op": "matmul", "m": 256, "n": 6144, "k": 4096, "out": "bf16"},
        # odd sizes, 32-bit output (logits, or a sum that goes on in 32 bits), K ends inside a scale block
        {"name": "matmul_odd_f32", "op": "matmul", "m": 333, "n": 1001, "k": 2000, "out": "f32"},
        # a prompt's projection to the keys and values of 32 heads
        {"name": "matmul_prompt", "op": "matmul", "m": 16384, "n": 8192, "k": 4096, "out": "bf16"},
        # short ragged prompts, some continuing a cached prefix
        {"name": "expanded_ragged", "op": "expanded", "seqs": 6, "tokens": 1500, "context": 700, "heads": 16},
        # one long prompt
        {"name": "expanded_long", "op": "expanded", "seqs": 1, "tokens": 8192, "context": 0, "heads": 32},
        # one user, a short conversation: latency
        {"name": "absorbed_single", "op": "absorbed", "seqs": 1, "queries": 1, "heads": 32, "len": 700, "page": 64, "empty": False},
        # drafted tokens verified three at a time, ragged, some sequences still without a cache
        {"name": "absorbed_draft", "op": "absorbed", "seqs": 37, "queries": 3, "heads": 16, "len": 3000, "page": 16, "empty": True},
        # a serving batch with long caches
        {"name": "absorbed_batch", "op": "absorbed", "seqs": 64, "queries": 1, "heads": 32, "len": 16384, "page": 64, "empty": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "matmul", "expanded", "absorbed"])
    if op == "norm":
        dim = _log_int(rng, 64, 8192)
        if rng.random() < 0.75:
            dim = max(16, dim // 16 * 16)
        tokens = _log_int(rng, 1, min(65536, (1 << 28) // dim))
        normed = rng.random() < 0.5
        return {"op": op, "tokens": tokens, "dim": dim, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "residual": rng.random() < 0.7, "normed": normed, "quant": not normed or rng.random() < 0.5}
    if op == "matmul":
        k = 16 * _log_int(rng, 8, 512)
        n = _log_int(rng, 64, 8192)
        m = _log_int(rng, 1, min(16384, 16384 * 8192 * 4096 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "bf16", "f32"])}
    if op == "expanded":
        heads = rng.choice([4, 7, 16, 32])
        tokens = _log_int(rng, 8, 6000)
        return {"op": op, "seqs": min(tokens, _log_int(rng, 1, 16)), "tokens": tokens,
                "context": rng.choice([0, 0, _log_int(rng, 1, 2000)]), "heads": heads}
    seqs = _log_int(rng, 1, 100)
    return {"op": op, "seqs": seqs, "queries": rng.choice([1, 1, 1, 2, 3, 4]), "heads": rng.choice([8, 16, 20, 32, 64, 128]),
            "len": _log_int(rng, 16, min(65536, 400000 // seqs)), "page": rng.choice([16, 32, 64, 128]),
            "empty": rng.random() < 0.3}


# ---------------------------------------------------------------- inputs
def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _ragged(case, seed):
    """(query lengths, key lengths) of a case, made from the seed alone: their spread, not their sum, follows the seed."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    n = case["seqs"]
    if case["op"] == "expanded":
        w = torch.rand(n, generator=g) + 0.1
        cut = (torch.cumsum(w, 0) / w.sum() * case["tokens"]).round().long()
        cut[-1] = case["tokens"]
        lq = torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long))
        extra = (torch.rand(n, generator=g) * 2 * case["context"]).long() if n > 1 else torch.full((1,), case["context"])
        extra[0] = case["context"] if n == 1 else 0
        return lq, lq + extra
    if n == 1:
        return None, torch.full((1,), case["len"])
    lk = (torch.rand(n, generator=g) * case["len"]).long() + 1
    lk[torch.randint(0, n, (1,), generator=g)] = case["len"]
    if case["empty"]:
        lk[torch.rand(n, generator=g) < 0.15] = 0
        lk[0], lk[-1] = 0, min(1, case["len"])
    return None, lk


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    s = dict(case)
    if case["op"] == "norm":
        t, d, dt = case["tokens"], case["dim"], _dtype(case["dtype"])
        # a residual stream: some channels far larger than the others, rows of different size
        chan = torch.exp(0.8 * normal(d, dtype=torch.float32))
        s["x"] = (normal(t, d, dtype=torch.float32) * chan).to(dt)
        s["residual_in"] = (3 * normal(t, d, dtype=torch.float32) * chan).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * normal(d, dtype=torch.float32)).to(dt)
        s["eps"] = 1e-6
    elif case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // 128), -(-n // 128)
        e4m3 = lambda r: (normal(r, k) * 112).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
        s["a"], s["b"] = e4m3(m), e4m3(n)
        s["a_scale"] = (torch.exp(0.5 * normal(m, kb, dtype=torch.float32)) / 112).contiguous()
        s["b_scale"] = (torch.exp(0.3 * normal(nb, kb, dtype=torch.float32)) / (112 * math.sqrt(k))).contiguous()
        s["out_dtype"] = _dtype(case["out"])
    elif case["op"] == "expanded":
        lq, lk = _ragged(case, seed)
        h, tq, tk = case["heads"], int(lq.sum()), int(lk.sum())
        s["q"] = normal(tq, h, NOPE + ROPE)
        s["kv"] = normal(tk, h, NOPE + VDIM)     # one projection's output: keys and values are views of it
        s["k_nope"], s["v"] = s["kv"][..., :NOPE], s["kv"][..., NOPE:]
        s["k_rope"] = normal(tk, ROPE)
        zero = torch.zeros(1, dtype=torch.long)
        s["cu_q"] = torch.cat([zero, lq.cumsum(0)]).to(DEV, torch.int32)
        s["cu_k"] = torch.cat([zero, lk.cumsum(0)]).to(DEV, torch.int32)
        s["max_q"], s["max_k"] = int(lq.max()), int(lk.max())
        s["scale"] = 1 / math.sqrt(NOPE + ROPE)
    else:
        _, lk = _ragged(case, seed)
        n, page = case["seqs"], case["page"]
        pages = (lk + page - 1) // page
        total, width = int(pages.sum()) + 3, max(1, int(pages.max()))
        gc = torch.Generator().manual_seed(seed + 5)
        order = torch.randperm(total, generator=gc)
        table = torch.zeros(n, width, dtype=torch.long)
        first = torch.cumsum(pages, 0) - pages
        used = torch.arange(width)[None] < pages[:, None]
        table[used] = order[(first[:, None] + torch.arange(width)[None])[used]]
        s["q"] = normal(n, case["queries"], case["heads"], RANK + ROPE)
        s["cache"] = normal(total, page, RANK + ROPE)
        s["table"] = table.to(DEV, torch.int32)
        s["lens"] = lk.to(DEV, torch.int32)
        s["max_len"] = max(1, int(lk.max()))
        s["scale"] = 1 / math.sqrt(NOPE + ROPE)
    return s


# ---------------------------------------------------------------- the pass
def _plain_norm(s):
    h = s["x"].float()
    if s["residual"]:
        h = h + s["residual_in"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    out = {"residual": h.to(s["x"].dtype) if s["residual"] else None, "normed": y.to(s["x"].dtype) if s["normed"] else None}
    if s["quant"]:
        t, d = y.shape
        kb = -(-d // 128)
        blocks = torch.nn.functional.pad(y, (0, kb * 128 - d)).view(t, kb, 128)
        amax = blocks.abs().amax(-1).clamp_min(1e-12)
        out["scales"] = amax / 448
        q = (blocks * (448 / amax)[..., None]).view(t, kb * 128)[:, :d]
        out["quantized"] = q.clamp(-448, 448).to(torch.float8_e4m3fn).contiguous()
    return out


def _plain_matmul(s):
    k, n = s["k"], s["n"]
    a = s["a"].float() * s["a_scale"].repeat_interleave(128, 1)[:, :k]
    b = s["b"].float() * s["b_scale"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return {"out": (a @ b.t()).to(s["out_dtype"])}


def _softmax_plain(scores, hidden):
    """exp(scores - max) with hidden places zero, its sum, and log-sum-exp; rows with nothing visible give zeros and -inf."""
    scores = scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total, (top + total.log()).squeeze(-1)


def _plain_expanded(s):
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    iq, ik = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    lq, lk = cq.diff(), ck.diff()
    at_q = (cq[:-1, None] + iq).clamp_max(s["q"].shape[0] - 1)               # [n, max_q]
    at_k = (ck[:-1, None] + ik).clamp_max(s["kv"].shape[0] - 1)
    q = s["q"][at_q].float().transpose(1, 2)                                # [n, h, max_q, 192]
    k = torch.cat([s["k_nope"][at_k], s["k_rope"][at_k][:, :, None].expand(-1, -1, s["heads"], -1)], -1).float().transpose(1, 2)
    v = s["v"][at_k].float().transpose(1, 2)
    hidden = ik[None, None] > iq[None, :, None] + (lk - lq)[:, None, None]
    hidden = hidden | (ik[None, None] >= lk[:, None, None])
    p, total, lse = _softmax_plain((q @ k.transpose(-1, -2)).mul_(s["scale"]), hidden[:, None])
    o = (p @ v / total.clamp_min(1e-30)).transpose(1, 2)                     # [n, max_q, h, 128]
    real = iq[None] < lq[:, None]
    return {"out": o[real].to(s["q"].dtype), "lse": lse.transpose(1, 2)[real]}


def _plain_absorbed(s):
    n, page = s["seqs"], s["page"]
    ik = torch.arange(s["max_len"], device=DEV)
    at = s["table"].long()[:, ik // page] * page + ik % page                 # [n, max_len]
    c = s["cache"].view(-1, RANK + ROPE)[at].float()                         # [n, max_len, 576]
    lq, h = s["queries"], s["heads"]
    q = s["q"].float().reshape(n, lq * h, RANK + ROPE)
    last = s["lens"].long()[:, None] - lq + torch.arange(lq, device=DEV)     # [n, lq] last visible key
    hidden = ik[None, None] > last[:, :, None]
    p, total, lse = _softmax_plain((q @ c.transpose(1, 2)).mul_(s["scale"]), hidden.repeat_interleave(h, 1))
    o = p @ c[..., :RANK] / total.clamp_min(1e-30)
    return {"out": o.view(n, lq, h, RANK).to(s["q"].dtype), "lse": lse.view(n, lq, h)}


def run(s):
    if own:
        import kda_gated_delta_chunked_gb300 as kda
        if s["op"] == "norm":
            y, q, sc, r = kda.rms_norm(s["x"], s["weight"], s["residual_in"], eps=s["eps"], normed=s["normed"], quantize=s["quant"])
            return {"residual": r, "normed": y, "quantized": q, "scales": sc}
        if s["op"] == "matmul":
            return {"out": kda.matmul_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=s["out_dtype"])}
        if s["op"] == "expanded":
            o, lse = kda.latent_prefill(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"], s["cu_k"], scale=s["scale"])
            return {"out": o, "lse": lse}
        o, lse = kda.latent_decode(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"])
        return {"out": o, "lse": lse}
    return {"norm": _plain_norm, "matmul": _plain_matmul, "expanded": _plain_expanded, "absorbed": _plain_absorbed}[s["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        t, d, e = case["tokens"], case["dim"], 2 if case["dtype"] == "bf16" else 4
        b = t * d * e + d * e
        b += 2 * t * d * e if case["residual"] else 0
        b += t * d * e if case["normed"] else 0
        b += t * d + 4 * t * -(-d // 128) if case["quant"] else 0
        return {"bytes": b, "flops": 5 * t * d}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // 128), -(-n // 128)
        return {"bytes": (m + n) * k + 4 * kb * (m + nb) + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    h = case["heads"]
    lq, lk = _ragged(case, 0)
    if case["op"] == "expanded":
        tq, tk = int(lq.sum()), int(lk.sum())
        pairs = int((lq * (lk - lq) + lq * (lq + 1) // 2).sum())
        b = 2 * (tq * h * (NOPE + ROPE) + tk * h * (NOPE + VDIM) + tk * ROPE + tq * h * VDIM) + 4 * tq * h
        return {"bytes": b, "flops": 2 * pairs * h * (NOPE + ROPE + VDIM)}
    n, q = case["seqs"], case["queries"]
    tk = int(lk.sum())
    b = 2 * (tk * (RANK + ROPE) + n * q * h * (2 * RANK + ROPE)) + 4 * n * q * h
    return {"bytes": b, "flops": 2 * tk * q * h * (2 * RANK + ROPE)}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    """Written row by row from the definitions, apart from the plain forms; a sequence at a time for the attentions."""
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "norm":
        t, d = case["tokens"], case["dim"]
        h = s["x"].to(f) + (s["residual_in"].to(f) if case["residual"] else 0)
        y = h / ((h * h).sum(1, keepdim=True) / d + s["eps"]).sqrt() * s["weight"].to(f)
        out = {"residual": h if case["residual"] else None, "normed": y if case["normed"] else None}
        if case["quant"]:
            size = torch.empty(t, -(-d // 128), dtype=f, device=DEV)
            whole = d // 128 * 128
            if whole:
                size[:, :d // 128] = y[:, :whole].reshape(t, -1, 128).abs().max(2).values
            if whole < d:
                size[:, -1] = y[:, whole:].abs().max(1).values
            size = torch.maximum(size, torch.tensor(1e-12, dtype=f, device=DEV)) / 448
            out["scales"] = size
            out["quantized"] = _nearest_e4m3(y / size.repeat_interleave(128, 1)[:, :d])
        return out
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        acc = torch.zeros(m, n, dtype=f, device=DEV)
        rows = torch.arange(n, device=DEV) // 128
        for j in range(-(-k // 128)):
            part = slice(128 * j, min(k, 128 * j + 128))
            acc.addmm_(s["a"][:, part].to(f) * s["a_scale"][:, j, None].to(f), (s["b"][:, part].to(f) * s["b_scale"][rows, j, None].to(f)).t())
        return {"out": acc}
    if case["op"] == "expanded":
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        out = torch.zeros(cq[-1], case["heads"], VDIM, dtype=f, device=DEV)
        lse = torch.full((cq[-1], case["heads"]), -math.inf, dtype=f, device=DEV)
        for i in range(case["seqs"]):
            lq, lk = cq[i + 1] - cq[i], ck[i + 1] - ck[i]
            seen = torch.tril(torch.ones(lq, lk, dtype=torch.bool, device=DEV), diagonal=lk - lq)
            for h in range(case["heads"]):
                q, ks = s["q"][cq[i]:cq[i + 1], h].to(f), slice(ck[i], ck[i + 1])
                x = q[:, :NOPE] @ s["k_nope"][ks, h].to(f).t() + q[:, NOPE:] @ s["k_rope"][ks].to(f).t()
                _attend(x * s["scale"], seen, s["v"][ks, h].to(f), out[cq[i]:cq[i + 1], h], lse[cq[i]:cq[i + 1], h])
        return {"out": out, "lse": lse}
    n, lq, h, page = case["seqs"], case["queries"], case["heads"], case["page"]
    out = torch.zeros(n, lq, h, RANK, dtype=f, device=DEV)
    lse = torch.full((n, lq, h), -math.inf, dtype=f, device=DEV)
    table, lens = s["table"].tolist(), s["lens"].tolist()
    for i in range(n):
        if lens[i] == 0:
            continue
        c = s["cache"][table[i][:-(-lens[i] // page)]].reshape(-1, RANK + ROPE)[:lens[i]].to(f)
        for j in range(lq):
            end = lens[i] - lq + 1 + j
            if end > 0:
                x = (s["q"][i, j].to(f) @ c[:end].t()) * s["scale"]
                _attend(x, torch.ones_like(x, dtype=torch.bool), c[:end, :RANK], out[i, j], lse[i, j])
    return {"out": out, "lse": lse}


def _attend(x, seen, v, out, lse):
    some = seen.any(1)
    x = torch.where(seen, x, torch.full_like(x, -math.inf))[some]
    lse[some] = torch.logsumexp(x, 1)
    out[some] = torch.softmax(x, 1) @ v


def _nearest_e4m3(x):
    """The e4m3 value nearest to each x (ties to even): 3 bits behind the leading one, the step 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)
