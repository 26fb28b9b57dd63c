"""Cases, plain forms and 64-bit definitions of the rotary positions and of the
quantised cache of latent attention.

The layers of full attention that a KDA stack alternates with keep, for each
token, one latent of 512 channels and one rotary key of 64, shared by the heads.
Serving them needs the rotary channels turned, the latents quantised as they are
written to the paged cache, read back where a prompt goes on behind a cached
prefix, and attention that reads the quantised cache:

  rotary  theta[t, i] = position[t] f[i]; pairs (a, b) of the rotated channels,
          neighbours or half of them apart, become scale (a cos - b sin, b cos + a sin);
          the gradient turns the other way
  write   e: the smallest integer with max |c| <= 448 2^e, within -100 .. 120;
          codes e4m3(c / 2^e), the rotary key in bf16, and the byte e + 127
  read    2^e code, and the rotary key
  decode  attention of one or a few tokens a sequence over that cache: keys
          [2^e code | rope], values 2^e code

A page holds its tokens' rows (512 codes, 64 bf16), then a byte of scale for each
token, padded to 128 bytes.  ``own`` selects between the plain form (elementary
torch operations) and the package's calls.
"""
import math

import torch

own = False

RANK, ROPE, ROW = 512, 64, 640
DEV = "cuda"


def listed():
    return [
        # one decoded token's queries (the last 64 of 192 channels of each head) and its shared key: latency alone
        {"name": "rotary_token", "op": "rotary", "tokens": 1, "heads": 32, "width": 192, "dim": 64, "offset": 128, "key": True,
         "dtype": "bf16", "interleaved": True, "inverse": False, "wide": False, "far": 100000, "scaled": True},
        # 32-bit activations, the first 48 of 80 channels, halves: a small model's odd batch
        {"name": "rotary_odd_f32", "op": "rotary", "tokens": 777, "heads": 7, "width": 80, "dim": 48, "offset": 0, "key": False,
         "dtype": "f32", "interleaved": False, "inverse": False, "wide": True, "far": 5000, "scaled": False},
        # a long prompt in a context of a million positions, frequencies scaled for it
        {"name": "rotary_prompt", "op": "rotary", "tokens": 32768, "heads": 32, "width": 192, "dim": 64, "offset": 128, "key": True,
         "dtype": "bf16", "interleaved": True, "inverse": False, "wide": False, "far": 1000000, "scaled": True},
        # the gradient of whole heads of 128 in training
        {"name": "rotary_gradient", "op": "rotary", "tokens": 8192, "heads": 16, "width": 128, "dim": 128, "offset": 0, "key": False,
         "dtype": "bf16", "interleaved": False, "inverse": True, "wide": False, "far": 8192, "scaled": False},
        # a decode step of 48 sequences: one new token each
        {"name": "write_step", "op": "write", "seqs": 48, "tokens": 48, "context": 3000, "dtype": "bf16", "page": 64},
        # ragged prompts behind what is cached already, pages of 16
        {"name": "write_prompts", "op": "write", "seqs": 21, "tokens": 65536, "context": 500, "dtype": "bf16", "page": 16},
        # a short prefix in 32 bits
        {"name": "read_odd_f32", "op": "read", "seqs": 3, "tokens": 1001, "context": 0, "dtype": "f32", "page": 32},
        # the cached prefixes of a batch that goes on
        {"name": "read_prefixes", "op": "read", "seqs": 16, "tokens": 100000, "context": 0, "dtype": "bf16", "page": 64},
        # one user, a short conversation: latency
        {"name": "decode_single", "op": "decode", "seqs": 1, "queries": 1, "heads": 32, "len": 700, "page": 64, "empty": False},
        # drafted tokens verified three at a time, ragged, some sequences still without a cache
        {"name": "decode_draft", "op": "decode", "seqs": 37, "queries": 3, "heads": 16, "len": 3001, "page": 16, "empty": True},
        # a serving batch with long caches
        {"name": "decode_batch", "op": "decode", "seqs": 64, "queries": 1, "heads": 32, "len": 16384, "page": 64, "empty": False},
        # many heads, a few long contexts
        {"name": "decode_heads", "op": "decode", "seqs": 9, "queries": 1, "heads": 128, "len": 30000, "page": 128, "empty": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "write", "read", "decode", "decode"])
    if op == "rotary":
        dim = rng.choice([16, 32, 48, 64, 64, 80, 96, 128, 2 * rng.randint(1, 64)])
        rest = rng.choice([0, 0, 16 * rng.randint(0, 8), rng.randint(1, 128)])
        heads, width = _log_int(rng, 1, 64), dim + rest
        tokens = _log_int(rng, 1, min(65536, 200000000 // (heads * width)))
        return {"op": op, "tokens": tokens, "heads": heads, "width": width, "dim": dim, "offset": rng.choice([0, rest]),
                "key": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "f32"]), "interleaved": rng.random() < 0.5,
                "inverse": rng.random() < 0.3, "wide": rng.random() < 0.4, "far": _log_int(rng, 1000, 2000000),
                "scaled": rng.random() < 0.5}
    if op in ("write", "read"):
        seqs = _log_int(rng, 1, 128)
        one = op == "write" and rng.random() < 0.3          # a step: one token each
        tokens = seqs if one else _log_int(rng, max(seqs, 4), 65536)
        return {"op": op, "seqs": seqs, "tokens": tokens, "context": 0 if op == "read" else _log_int(rng, 1, 2000),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "page": rng.choice([16, 32, 64, 128])}
    seqs = _log_int(rng, 1, 100)
    return {"op": op, "seqs": seqs, "queries": rng.choice([1, 1, 1, 2, 3, 4]), "heads": rng.choice([8, 16, 20, 32, 64, 128]),
            "len": _log_int(rng, 16, min(65536, 400000 // seqs)), "page": rng.choice([16, 32, 64, 128]),
            "empty": rng.random() < 0.3}


# ---------------------------------------------------------------- inputs
def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _page_bytes(page):
    return -(-page * (ROW + 1) // 128) * 128


def _views(cache, page):
    """The codes, rotary keys and scale bytes of a cache, as views of it."""
    rows = cache[:, :page * ROW].unflatten(1, (page, ROW))
    return rows[..., :RANK].view(torch.float8_e4m3fn), rows[..., RANK:].view(torch.bfloat16), cache[:, page * ROW:page * (ROW + 1)]


def _quantise(c):
    """(codes, scale bytes) of latents [..., 512] in 32 bits."""
    m, k = torch.frexp(c.abs().amax(-1))                       # max = m 2^k, 1/2 <= m < 1; 448 = 7/8 2^9
    e = torch.where(m <= 0.875, k - 9, k - 8)
    e = torch.where(m == 0, torch.full_like(e, -100), e).clamp(-100, 120)
    return torch.ldexp(c, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _lengths(case, seed):
    """(new tokens, cached tokens) of each sequence on the host, made from the seed alone."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    n = case["seqs"]
    if case["op"] == "decode":
        if n == 1:
            return None, torch.full((1,), case["len"])
        lk = (torch.rand(n, generator=g) * case["len"]).long() + 1
        lk[torch.randint(0, n, (1,), generator=g)] = case["len"]
        if case["empty"]:
            lk[torch.rand(n, generator=g) < 0.15] = 0
            lk[0], lk[-1] = 0, min(1, case["len"])
        return None, lk
    if case["op"] == "write" and case["tokens"] == n:
        new = torch.ones(n, dtype=torch.long)
    else:
        w = torch.rand(n, generator=g) + 0.05
        cut = (torch.cumsum(w, 0) / w.sum() * case["tokens"]).round().long()
        cut[-1] = case["tokens"]
        new = torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long))
    return new, new + (torch.rand(n, generator=g) * 2 * case["context"]).long()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    s = dict(case)
    if case["op"] == "rotary":
        t, d, dt = case["tokens"], case["dim"], _dtype(case["dtype"])
        s["x"] = normal(t, case["heads"], case["width"], dtype=dt)
        s["key_in"] = normal(t, d, dtype=dt) if case["key"] else None
        # consecutive positions of a few sequences, each from a place of its own
        gc = torch.Generator().manual_seed(seed + 3)
        n = min(t, 5)
        starts = (torch.rand(n, generator=gc) * case["far"]).long()
        at = torch.arange(t)
        per = -(-t // n)
        s["positions"] = (starts[(at // per).clamp_max(n - 1)] + at % per).to(DEV, torch.int64 if case["wide"] else torch.int32)
        f = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
        s["scale"] = 1.0
        if case["scaled"]:      # for 32 times the trained length: fast pairs as they are, slow ones 32 times slower
            turns = 4096 * f / (2 * math.pi)
            keep = ((turns - 1) / 31).clamp(0, 1)
            f = f * (keep + (1 - keep) / 32)
            s["scale"] = 0.1 * math.log(32) + 1
        s["frequencies"] = f.to(DEV)
        return s
    new, cached = _lengths(case, seed)
    n, page = case["seqs"], case["page"]
    pages = (cached + page - 1) // page
    total, width = int(pages.sum()) + 3, max(1, int(pages.max()))
    if case["op"] == "write":                                  # a pool of pages for the longest contexts
        total = (case["tokens"] + 2 * case["context"] * n) // page + n + 3
    gc = torch.Generator().manual_seed(seed + 5)
    order = torch.randperm(total, generator=gc)
    table = torch.zeros(n, width, dtype=torch.long)
    first = torch.cumsum(pages, 0) - pages
    used = torch.arange(width)[None] < pages[:, None]
    table[used] = order[(first[:, None] + torch.arange(width)[None])[used]]
    s["table"] = table.to(DEV, torch.int32)
    s["lens"] = cached.to(DEV, torch.int32)
    # latents behind their norm: some channels larger than others, tokens of different size
    chan = torch.exp(0.5 * normal(RANK, dtype=torch.float32))
    s["cache"] = torch.zeros(total, _page_bytes(page), dtype=torch.uint8, device=DEV)
    codes, rope, scales = _views(s["cache"], page)
    for p in range(0, total, 65536 // page):                   # in slices: the 32-bit latents are the larger part
        q = slice(p, min(total, p + 65536 // page))
        size = torch.exp(0.4 * normal(q.stop - p, page, 1, dtype=torch.float32))
        c, b = _quantise(normal(q.stop - p, page, RANK, dtype=torch.float32) * chan * size)
        codes[q], scales[q] = c, b
        rope[q] = normal(q.stop - p, page, ROPE)
    if case["op"] == "decode":
        s["q"] = normal(n, case["queries"], case["heads"], RANK + ROPE)
        s["max_len"] = max(1, int(cached.max()))
        s["softmax_scale"] = 1 / math.sqrt(128 + ROPE)
        return s
    t, dt = case["tokens"], _dtype(case["dtype"])
    s["cu"] = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)]).to(DEV, torch.int32)
    if case["op"] == "write":
        s["steps"] = t == n
        # one projection's output: the latent and the rotary key are views of it
        both = normal(t, RANK + ROPE, dtype=torch.float32)
        both[:, :RANK] *= chan * torch.exp(0.4 * normal(t, 1, dtype=torch.float32))
        both = both.to(dt)
        s["latent"], s["rope"] = both[:, :RANK], both[:, RANK:]
    return s


# ---------------------------------------------------------------- the pass
def _plain_turn(x, cos, sin, s):
    """The rotated channels x [t, h, d] in 32 bits, cos and sin [t, 1, d / 2]."""
    if s["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_rotary(s):
    theta = s["positions"].double()[:, None] * s["frequencies"]
    if s["inverse"]:
        theta = -theta
    cos, sin = (theta.cos() * s["scale"]).float()[:, None], (theta.sin() * s["scale"]).float()[:, None]
    y = s["x"].clone()
    part = slice(s["offset"], s["offset"] + s["dim"])
    y[..., part] = _plain_turn(s["x"][..., part].float(), cos, sin, s).to(y.dtype)
    key = s["key_in"]
    return {"out": y, "key": None if key is None else _plain_turn(key[:, None].float(), cos, sin, s)[:, 0].to(key.dtype)}


def _places(s):
    """Row in the flattened cache of every token of the packed rows."""
    t, page, cu = s["tokens"], s["page"], s["cu"].long()
    at = torch.arange(t, device=DEV)
    seq = torch.bucketize(at, cu[1:], right=True)
    place = s["lens"].long()[seq] - cu[seq + 1] + at
    return s["table"].long()[seq, place // page], place % page


def _plain_write(s):
    codes, rope, scales = _views(s["cache"], s["page"])
    at = _places(s)
    c, b = _quantise(s["latent"].float())
    codes.view(torch.uint8)[at] = c.view(torch.uint8)
    rope[at] = s["rope"].to(torch.bfloat16)
    scales[at] = b
    return {"codes": codes, "rope": rope, "scales": scales}


def _plain_read(s):
    codes, rope, scales = _views(s["cache"], s["page"])
    at = _places(s)
    c = codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    dt = _dtype(s["dtype"])
    return {"latent": torch.ldexp(c, scales[at].int()[:, None] - 127).to(dt), "rope": rope[at].to(dt)}


def _plain_decode(s):
    n, page = s["seqs"], s["page"]
    codes, rope, scales = _views(s["cache"], page)
    ik = torch.arange(s["max_len"], device=DEV)
    at = s["table"].long()[:, ik // page], (ik % page).expand(n, -1)          # [n, max_len]
    v = torch.ldexp(codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float(), scales[at].int()[..., None] - 127)
    lq, h = s["queries"], s["heads"]
    q = s["q"].float().reshape(n, lq * h, RANK + ROPE)
    scores = (q[..., :RANK] @ v.transpose(1, 2) + q[..., RANK:] @ rope[at].float().transpose(1, 2)).mul_(s["softmax_scale"])
    last = s["lens"].long()[:, None] - lq + torch.arange(lq, device=DEV)      # [n, lq] last visible token
    hidden = ik[None, None] > last[:, :, None]
    scores = scores.masked_fill_(hidden.repeat_interleave(h, 1), -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p @ v / total.clamp_min(1e-30)
    return {"out": o.view(n, lq, h, RANK).to(s["q"].dtype), "lse": (top + total.log()).view(n, lq, h)}


def run(s):
    if own:
        import kda_gated_delta_chunked_gb300 as kda
        if s["op"] == "rotary":
            y, k = kda.rotary(s["x"], s["positions"], s["frequencies"], key=s["key_in"], offset=s["offset"],
                              interleaved=s["interleaved"], inverse=s["inverse"], scale=s["scale"])
            return {"out": y, "key": k}
        if s["op"] == "write":
            kda.latent_cache_write(s["latent"], s["rope"], s["cache"], s["table"], s["lens"], None if s["steps"] else s["cu"],
                                   page_size=s["page"])
            return dict(zip(("codes", "rope", "scales"), _views(s["cache"], s["page"])))
        if s["op"] == "read":
            c, r = kda.latent_cache_read(s["cache"], s["table"], s["lens"], s["cu"], total_tokens=s["tokens"],
                                         page_size=s["page"], rank=RANK, d_rope=ROPE, dtype=_dtype(s["dtype"]))
            return {"latent": c, "rope": r}
        o, lse = kda.latent_decode(s["q"], s["cache"], s["table"], s["lens"], scale=s["softmax_scale"], rank=RANK,
                                   page_size=s["page"])
        return {"out": o, "lse": lse}
    return {"rotary": _plain_rotary, "write": _plain_write, "read": _plain_read, "decode": _plain_decode}[s["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "rotary":
        t, h, w, d = case["tokens"], case["heads"], case["width"], case["dim"]
        e = 2 if case["dtype"] == "bf16" else 4
        keys = d if case["key"] else 0
        return {"bytes": 2 * t * (h * w + keys) * e + t * (8 if case["wide"] else 4) + 4 * d, "flops": 3 * t * (h * d + keys)}
    if case["op"] in ("write", "read"):
        e = 2 if case["dtype"] == "bf16" else 4
        t = case["tokens"]
        return {"bytes": t * ((RANK + ROPE) * e + ROW + 1) + 4 * (2 * case["seqs"] + 1) + 4 * -(-t // case["page"]), "flops": 2 * t * RANK}
    _, lk = _lengths(case, 0)
    n, q, h, tk = case["seqs"], case["queries"], case["heads"], int(lk.sum())
    b = tk * (ROW + 1) + 2 * n * q * h * (2 * RANK + ROPE) + 4 * n * q * h + 4 * -(-tk // case["page"])
    return {"bytes": b, "flops": 2 * tk * q * h * (2 * RANK + ROPE)}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    """Written from the definitions, apart from the plain forms: rotations as complex products, tokens and sequences one
    after another."""
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "rotary":
        d, o = case["dim"], case["offset"]
        turn = torch.polar(torch.tensor(s["scale"], dtype=f, device=DEV), s["positions"].to(f)[:, None] * s["frequencies"])
        turn = (turn.conj() if case["inverse"] else turn)[:, None]

        def rotated(x):                                         # [t, h, d]
            x = x.to(f)
            pairs = x.unflatten(-1, (d // 2, 2)) if case["interleaved"] else x.unflatten(-1, (2, d // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            return (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        y = s["x"].to(f)
        y[..., o:o + d] = rotated(s["x"][..., o:o + d])
        return {"out": y, "key": None if s["key_in"] is None else rotated(s["key_in"][:, None])[:, 0]}
    page, table, lens = case["page"], s["table"].tolist(), s["lens"].tolist()
    codes, rope, scales = _views(s["cache"], page)
    if case["op"] in ("write", "read"):
        cu, rows = s["cu"].tolist(), []
        for i in range(case["seqs"]):
            new = cu[i + 1] - cu[i]
            rows += [table[i][p // page] * page + p % page for p in range(lens[i] - new, lens[i])]
        rows = torch.tensor(rows, device=DEV)
        v, r, b = codes.to(f).flatten(0, 1), rope.to(f).flatten(0, 1), scales.reshape(-1).clone()
        if case["op"] == "read":
            return {"latent": v[rows] * torch.exp2(b[rows].to(f) - 127)[:, None], "rope": r[rows]}
        c = s["latent"].to(f)
        size = c.abs().max(1).values / 448
        e = torch.ceil(torch.log2(size.clamp_min(2.0 ** -100)))
        e = torch.where(torch.exp2(e - 1) >= size, e - 1, e)    # (the logarithm's rounding at powers of two)
        e = torch.where(torch.exp2(e) < size, e + 1, e).clamp(-100, 120)
        v[rows] = _nearest_e4m3(c / torch.exp2(e)[:, None])
        r[rows] = s["rope"].to(f)
        b[rows] = (e + 127).to(torch.uint8)
        shape = scales.shape
        return {"codes": v.view(*shape, RANK), "rope": r.view(*shape, ROPE), "scales": b.view(shape)}
    n, lq, h = case["seqs"], case["queries"], case["heads"]
    out = torch.zeros(n, lq, h, RANK, dtype=f, device=DEV)
    lse = torch.full((n, lq, h), -math.inf, dtype=f, device=DEV)
    for i in range(n):
        if lens[i] == 0:
            continue
        at = torch.tensor(table[i][:-(-lens[i] // page)], device=DEV)
        c = (codes[at].to(f) * torch.exp2(scales[at].to(f) - 127)[..., None]).flatten(0, 1)
        k = torch.cat([c, rope[at].to(f).flatten(0, 1)], 1)
        for j in range(lq):
            end = lens[i] - lq + 1 + j
            if end > 0:
                x = (s["q"][i, j].to(f) @ k[:end].t()) * s["softmax_scale"]
                lse[i, j] = torch.logsumexp(x, 1)
                out[i, j] = torch.softmax(x, 1) @ c[:end]
    return {"out": out, "lse": lse}


def _nearest_e4m3(x):
    """The e4m3 value nearest to each x (ties to even): 3 bits behind the leading one, the step 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)
