"""The attention half of a decoder block over a 4-bit paged cache, and the scores of its tokens.

Three groups of calls are stood for here, each in a plain torch form and, where
``own`` is true, as the calls of ``block_quantized_moe_layer_gb300``:

``append``  the step before attention: RMS norm of every query and key head,
            rotation of their first ``rot`` channels, queries rounded to the
            activation type, keys and values quantised to 4 bits and stored in
            the pages the slots name; the stored rows are read back as values.
``attend``  causal attention of the last tokens of each sequence over that cache.
``score``   log probabilities of given tokens, the entropy of each row and its
            most probable alternatives.

The cache.  A page holds P tokens.  For each key/value head it holds four
arrays in turn: key codes [P][D/2], key scales [P][D/16], value codes and value
scales of the same shapes.  16 consecutive channels share a scale byte: the top
eight bits below the sign of a half-precision number d (5 exponent bits, 3
fraction bits), at most 896.  A channel is (c - 8) d for its code c in 0..15;
channel e of each eight is nibble e/2 + 4 (e%2) of their 32-bit word.  Storing
takes d = amax/7 rounded to nearest even, c = 8 + x/d rounded to nearest even
and clamped.
"""
import math

import torch

own = False

_ORDER = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble of channel e of eight
_HEADS = {  # name: (query heads, key/value heads, channels, rotated channels)
    "64x4x192": (64, 4, 192, 64),
    "32x8x128": (32, 8, 128, 128),
    "16x16x64": (16, 16, 64, 32),
    "16x2x256": (16, 2, 256, 64),
}


def listed():
    return [
        # one verify batch (a token and three drafts): what every round of one user pays
        dict(name="append_verify", op="append", heads="64x4x192", tokens=4, far=30000, page=64, act="bf16"),
        # 32 users' verify batches at once, every channel rotated, small pages
        dict(name="append_batch", op="append", heads="32x8x128", tokens=128, far=8192, page=16, act="bf16"),
        # a long prompt's chunk
        dict(name="append_prompt", op="append", heads="64x4x192", tokens=4096, far=20000, page=64, act="bf16"),
        # the smallest call: one token of one user with a short history, odd length
        dict(name="attend_token", op="attend", heads="64x4x192", seqs=1, tokens=1, length=257, window=0, page=64, act="bf16"),
        # one verify batch over a long history that ends inside a page
        dict(name="attend_verify_long", op="attend", heads="64x4x192", seqs=1, tokens=4, length=32765, window=0, page=64, act="bf16"),
        # 32 users, one token each, ragged histories, small pages
        dict(name="attend_batch", op="attend", heads="32x8x128", seqs=32, tokens=1, length=8192, window=0, page=16, act="bf16"),
        # 16 users' verify batches in a sliding-window layer
        dict(name="attend_window", op="attend", heads="64x4x192", seqs=16, tokens=4, length=8000, window=512, page=64, act="bf16"),
        # one ubatch of a prompt behind an earlier part of it
        dict(name="attend_prompt", op="attend", heads="64x4x192", seqs=1, tokens=1024, length=8192, window=0, page=64, act="bf16"),
        # the fp32 check mode
        dict(name="attend_check", op="attend", heads="16x16x64", seqs=2, tokens=3, length=999, window=0, page=32, act="f32"),
        # a verify batch's rows with the alternatives an API returns
        dict(name="score_verify", op="score", rows=4, vocab=32768, top=8, logits="f32"),
        # every token of a prompt
        dict(name="score_prompt", op="score", rows=1023, vocab=32768, top=5, logits="f32"),
        # a batch of users with a large vocabulary, bf16 logits
        dict(name="score_batch", op="score", rows=33, vocab=151936, top=20, logits="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "score"])
    if op == "append":
        return dict(op=op, heads=rng.choice(sorted(_HEADS)), tokens=_log(rng, 1, 4096), far=_log(rng, 5000, 60000),
                    page=rng.choice([16, 32, 64, 128]), act=rng.choice(["bf16", "bf16", "f32"]))
    if op == "score":
        rows = _log(rng, 1, 1024)
        return dict(op=op, rows=rows, vocab=_log(rng, 1000, min(200000, 33500000 // rows)), top=rng.randint(0, 20),
                    logits=rng.choice(["f32", "bf16"]))
    heads, page = rng.choice(sorted(_HEADS)), rng.choice([16, 32, 64, 128])
    kind = rng.choice(["small", "small", "small", "prompt", "check"])
    if kind == "small":  # single tokens and verify batches
        seqs = _log(rng, 1, 32)
        return dict(op=op, heads=heads, seqs=seqs, tokens=rng.randint(1, 8), length=_log(rng, 16, 65536 // seqs),
                    window=rng.choice([0, 0, 512, 100]), page=page, act="bf16")
    if kind == "prompt":
        seqs = rng.randint(1, 3)
        tokens = _log(rng, 9, 1024 // seqs)
        return dict(op=op, heads=heads, seqs=seqs, tokens=tokens, length=tokens + _log(rng, 1, 7000), window=rng.choice([0, 0, 512]),
                    page=page, act="bf16")
    return dict(op=op, heads=heads, seqs=rng.randint(1, 4), tokens=rng.randint(1, 4), length=_log(rng, 16, 2000), window=0, page=page,
                act="f32")


# ------------------------------------------------------------------ shapes


def _lengths(case):
    """(tokens in the cache, new tokens among them) of each sequence: the first has the case's own, the others fewer."""
    n, t, lens, news = case["length"], case["tokens"], [], []
    for b in range(case["seqs"]):
        lens.append(max(1, n - (b * 2654435761 % 1000003) * n // 2 // 1000003))
        news.append(max(1, min(lens[-1], t if t <= 8 else t - b * t // 5)))
    return lens, news


def _visible(case):
    """Pairs of a query token and a cached token that it sees, and cached tokens that are seen, over all sequences."""
    pairs = seen = 0
    w = case["window"] or 1 << 40
    for n, t in zip(*_lengths(case)):
        pairs += sum(min(p + 1, w) for p in range(n - t, n))
        seen += min(n, t - 1 + w)
    return pairs, seen


def work(case):
    if case["op"] == "score":
        n, v = case["rows"], case["vocab"]
        return {"bytes": n * v * (4 if case["logits"] == "f32" else 2) + n * (4 + 8 + 8 * case["top"]), "flops": 5 * n * v}
    hq, hk, d, _ = _HEADS[case["heads"]]
    size = 2 if case["act"] == "bf16" else 4
    row = hk * d * 2 * 9 // 16  # a token's keys and values in the cache
    if case["op"] == "append":
        t = case["tokens"]
        return {"bytes": t * ((2 * hq + 2 * hk) * d * size + row + 2 * hk * d * 2 + 12), "flops": t * (hq + hk) * d * 7}
    pairs, seen = _visible(case)
    t = sum(_lengths(case)[1])
    return {"bytes": seen * row + 2 * t * hq * d * size, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ the cache in plain torch


def _arrays(pages, hk, p, d):
    """The four arrays of the page pool, as views: key codes, key scales, value codes, value scales."""
    n = pages.shape[0]
    at, out = 0, []
    rows = pages.view(n, hk, p * d * 9 // 8)
    for width in (d // 2, d // 16, d // 2, d // 16):
        out.append(rows[:, :, at:at + p * width].unflatten(2, (p, width)))
        at += p * width
    return out


def _quantise(x):
    """Codes packed in bytes [..., D/2] and scale bytes [..., D/16] of rows x [..., D]."""
    g = x.unflatten(-1, (-1, 16))
    v = g.abs().amax(-1) / 7
    step = torch.exp2((torch.frexp(v).exponent - 1).clamp(min=-14).to(v.dtype) - 3)
    d = (torch.round(v / step) * step).clamp(max=896.0)
    c = torch.where(d[..., None] > 0, torch.round(g / d[..., None]).clamp(-8, 7), torch.zeros_like(g)) + 8
    c = c.to(torch.uint8).flatten(-2).unflatten(-1, (-1, 8))
    nib = torch.empty_like(c)
    nib[..., _ORDER] = c
    packed = (nib[..., 0::2] | (nib[..., 1::2] << 4)).flatten(-2)
    return packed, (d.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)


def _values(codes, scales):
    """The fp32 rows [..., D] that codes [..., D/2] and scale bytes [..., D/16] stand for."""
    b = codes.unflatten(-1, (-1, 4))
    nib = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    c = nib[..., _ORDER].flatten(-2).unflatten(-1, (-1, 16)).to(torch.float32) - 8
    d = (scales.to(torch.int16) << 7).view(torch.float16).to(torch.float32)
    return (c * d[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case=case)
    if case["op"] == "score":
        # logits as a trained head gives them: a few likely tokens over a broad rest
        x = normal(case["rows"], case["vocab"]) * 2
        x += 6 * (torch.rand(x.shape, generator=gen, device="cuda") < 5.0 / case["vocab"])
        s["logits"] = x if case["logits"] == "f32" else x.to(torch.bfloat16)
        s["tokens"] = torch.randint(case["vocab"], (case["rows"],), generator=gen, device="cuda", dtype=torch.int32)
        return s
    hq, hk, d, rot = _HEADS[case["heads"]]
    page, dtype = case["page"], torch.bfloat16 if case["act"] == "bf16" else torch.float32
    per_page = hk * page * d * 9 // 8
    if case["op"] == "append":
        t = case["tokens"]
        # one projection's output: queries, keys and values of a token side by side
        s["qkv"] = (normal(t, (hq + 2 * hk) * d) * torch.exp(0.5 * normal(t, 1))).to(dtype)
        s["q_norm"], s["k_norm"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        first = int(torch.randint(case["far"] - t, (1,), generator=gen, device="cuda"))
        s["positions"] = torch.arange(first, first + t, device="cuda", dtype=torch.int32)
        n_pages = -(-t // page) + 3
        s["pages"] = torch.zeros(n_pages, per_page, dtype=torch.uint8, device="cuda")
        order = torch.randperm(n_pages, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda") + first % page
        s["slots"] = order[at // page] * page + at % page
        # a user keeps the angles' table; the plain form's in 64 bits, since positions reach far
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(case["far"], dtype=torch.float64, device="cuda")[:, None] * freq
        s["cos"], s["sin"] = angle.cos(), angle.sin()
        sizes = dict(n_pages=n_pages, T_max=t, S_max=1, len_max=case["far"])
    else:
        lens, news = _lengths(case)
        tables = [-(-n // page) for n in lens]
        n_pages = sum(tables) + 2
        s["pages"] = torch.empty(n_pages, per_page, dtype=torch.uint8, device="cuda")
        kc, ks, vc, vs = _arrays(s["pages"], hk, page, d)
        part = max(1, (1 << 26) // (hk * page * d))
        for at in range(0, n_pages, part):
            n = min(part, n_pages - at)
            for codes, scales in ((kc, ks), (vc, vs)):
                codes[at:at + n], scales[at:at + n] = _quantise(normal(n, hk, page, d))
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros(len(lens), max(tables), dtype=torch.int32)
        used = 0
        order_host = order.cpu()
        for b, n in enumerate(tables):
            table[b, :n] = order_host[used:used + n]
            used += n
        s["table"] = table.cuda()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = [0]
        for t in news:
            starts.append(starts[-1] + t)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["q"] = (normal(starts[-1], hq, d) * 1.5).to(dtype)
        s["max_q"], s["max_len"] = max(news), max(lens)
        sizes = dict(n_pages=n_pages, T_max=starts[-1], S_max=len(lens), len_max=max(lens))
    if own:
        import block_quantized_moe_layer_gb300 as pkg
        s["attention"] = pkg.Attention(hq, hk, d, page, act=pkg.ACT_BF16 if case["act"] == "bf16" else pkg.ACT_F32, rot_dim=rot,
                                       q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), window=case.get("window", 0), **sizes)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return {"append": _append, "attend": _attend, "score": _score}[s["case"]["op"]](s)


def _append(s):
    case = s["case"]
    hq, hk, d, rot = _HEADS[case["heads"]]
    t, p = case["tokens"], case["page"]
    q, k, v = s["qkv"].unflatten(1, (-1, d)).split([hq, hk, hk], 1)
    if own:
        rows = s["attention"].append(q, k, v, s["positions"], s["slots"], s["pages"])
        keys, values = s["attention"].read(s["slots"], s["pages"])
        return {"q": rows, "k": keys, "v": values}

    def normed(x, w, kind):
        x = x.to(kind)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.to(kind)
        c, n = s["cos"][s["positions"]].to(kind)[:, None], s["sin"][s["positions"]].to(kind)[:, None]
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * c - b * n, b * c + a * n, x[..., rot:]], -1)

    rows = normed(q, s["q_norm"], torch.float32).to(q.dtype)
    page, at = s["slots"] // p, s["slots"] % p
    kc, ks, vc, vs = _arrays(s["pages"], hk, p, d)
    # 64 bits: a value next to the border of two codes takes the nearer one
    kc[page, :, at], ks[page, :, at] = _quantise(normed(k, s["k_norm"], torch.float64))
    vc[page, :, at], vs[page, :, at] = _quantise(v.to(torch.float64))
    keys, values = _values(kc[page, :, at], ks[page, :, at]), _values(vc[page, :, at], vs[page, :, at])
    return {"q": rows, "k": keys.to(torch.bfloat16), "v": values.to(torch.bfloat16)}


def _attend(s):
    case = s["case"]
    if own:
        return s["attention"].forward(s["q"], s["pages"], s["starts"], s["lens"], s["table"], s["max_q"], s["max_len"])
    hq, hk, d, _ = _HEADS[case["heads"]]
    p, g = case["page"], hq // hk
    n = -(-s["max_len"] // p)

    def rows(codes, scales):  # [sequence, head, token, channel] of the sequences' pages in order
        pick = s["table"][:, :n].long()
        return _values(codes[pick], scales[pick]).permute(0, 2, 1, 3, 4).flatten(2, 3)

    kc, ks, vc, vs = _arrays(s["pages"], hk, p, d)
    news = s["starts"][1:] - s["starts"][:-1]
    at = s["starts"][:-1, None] + torch.arange(s["max_q"], device="cuda")
    q = s["q"][at.clamp(max=s["q"].shape[0] - 1).long()].to(torch.float32)  # [sequence, token, query head, channel]
    q = q.unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = q @ rows(kc, ks).transpose(2, 3) * d ** -0.5
    where = (s["lens"] - news)[:, None] + torch.arange(s["max_q"], device="cuda")
    key = torch.arange(n * p, device="cuda")
    sees = (key <= where[..., None]) & (key < s["lens"][:, None, None])
    if case["window"]:
        sees &= key > where[..., None] - case["window"]
    sees = sees[:, None].repeat(1, 1, g, 1)
    scores = scores.masked_fill_(~sees, -math.inf)
    scores = (scores - scores.amax(-1, keepdim=True)).exp_()
    out = (scores @ torch.where(key[:, None] < s["lens"][:, None, None, None], rows(vc, vs), 0.0)) / scores.sum(-1, keepdim=True)
    out = out.unflatten(2, (g, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return out[torch.arange(s["max_q"], device="cuda") < news[:, None]].to(s["q"].dtype)


def _score(s):
    top = s["case"]["top"]
    if own:
        import block_quantized_moe_layer_gb300 as pkg
        r = pkg.token_logprobs(s["logits"], s["tokens"], n_top=top)
        return [r["logprob"], r["entropy"], r["top_ids"], r["top_logprobs"]]
    x = s["logits"].to(torch.float32)
    most = x.amax(1, keepdim=True)
    z = x - most
    e = z.exp()
    total = e.sum(1, dtype=torch.float64)
    lse = total.log()
    entropy = lse - (e * z).sum(1, dtype=torch.float64) / total
    picked = z.gather(1, s["tokens"][:, None].long())[:, 0] - lse
    best, ids = torch.sort(x, dim=1, descending=True, stable=True)
    return [picked.float(), entropy.float(), ids[:, :top].to(torch.int32), (best[:, :top] - most - lse[:, None]).float()]


# ------------------------------------------------------------------ from the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "score":
        return _exact_score(s, case["top"])
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_score(s, top):
    x = s["logits"].double()
    logp = torch.log_softmax(x, 1)
    entropy = -(logp.exp() * logp).sum(1)
    rows = torch.arange(x.shape[0], device="cuda")
    taken = []
    rest = x.clone()
    for _ in range(top):  # the largest, the lowest index among equals, then the next
        j = (rest == rest.amax(1, keepdim=True)).to(torch.uint8).argmax(1)
        taken.append(j)
        rest[rows, j] = -math.inf
    ids = torch.stack(taken, 1) if top else rows.new_zeros(len(rows), 0)
    return [logp[rows, s["tokens"].long()], entropy, ids.to(torch.int32), logp.gather(1, ids)]


def _nearest(x, grid):
    """The entry of the ascending `grid` nearest to each x, the one at an even place where two are as near."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    a, b = x - grid[lo], grid[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _exact_append(s):
    case = s["case"]
    hq, hk, d, rot = _HEADS[case["heads"]]
    x = s["qkv"].double().view(case["tokens"], -1, d)
    where = s["positions"].double()[:, None]
    turn = torch.polar(torch.ones_like(where), where * 10000.0 ** (-2.0 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / rot))

    def turned(y, w):
        y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + 1e-6) * w.double()
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn[:, None]
        return torch.cat([z.real, z.imag, y[..., rot:]], -1)

    scale = torch.arange(199, device="cuda")  # every scale byte, and the scale it stands for
    e, m = scale // 8, (scale % 8).double()
    grid = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 15).double()), m / 8 * 2.0 ** -14)
    whole = torch.arange(-8, 8, device="cuda", dtype=torch.float64)

    def stored(y):
        y = y.unflatten(-1, (-1, 16))
        step = grid[_nearest(y.abs().amax(-1) / 7, grid)][..., None]
        return (whole[_nearest(torch.where(step > 0, y / step, 0.0), whole)] * step).flatten(-2)

    return {"q": turned(x[:, :hq], s["q_norm"]), "k": stored(turned(x[:, hq:hq + hk], s["k_norm"])), "v": stored(x[:, hq + hk:])}


def _exact_attend(s):
    case = s["case"]
    hq, hk, d, _ = _HEADS[case["heads"]]
    p, g = case["page"], hq // hk
    pool = s["pages"].view(-1, hk, p * d * 9 // 8)
    q = s["q"].double()
    out = torch.zeros_like(q)
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    for b, n in enumerate(lens):
        first, last = starts[b], starts[b + 1]
        mine = pool[s["table"][b, :-(-n // p)].long()]
        for h in range(hk):
            both = []
            for at in (0, p * d * 9 // 16):
                words = mine[:, h, at:at + p * d // 2].contiguous().view(torch.int32)
                scales = mine[:, h, at + p * d // 2:at + p * d * 9 // 16].long().reshape(-1, d // 16)[:n]
                codes = torch.stack([(words >> (4 * (e // 2 + 4 * (e % 2)))) & 15 for e in range(8)], -1).reshape(-1, d)[:n]
                e, m = scales // 8, (scales % 8).double()
                step = torch.where(e > 0, (8 + m) * torch.exp2((e - 18).double()), m * 2.0 ** -17)
                both.append((codes.double() - 8) * step.repeat_interleave(16, 1))
            keys, values = both
            where = torch.arange(n - (last - first), n, device="cuda")[:, None]
            key = torch.arange(n, device="cuda")
            hidden = key > where
            if case["window"]:
                hidden |= key <= where - case["window"]
            for i in range(h * g, (h + 1) * g):
                w = (q[first:last, i] @ keys.T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                out[first:last, i] = torch.softmax(w, 1) @ values
    return out
