"""A verify step over a tree of drafted tokens: attention, acceptance by chance, and the cache rows that stay.

Three groups of calls are stood for here, each in a plain torch form and, where
``own`` is true, as the calls of ``block_quantized_moe_layer_gb300``:

``tree``    attention of each sequence's last tokens, which are the nodes of a
            tree of drafts: a node sees the tokens before the tree and its own
            ancestors, over a 4-bit paged cache.
``verify``  the walk down the tree: drafts are accepted against the target's
            probabilities by given random numbers, and the next token is drawn
            from what the rejected ones leave.
``commit``  the accepted nodes' cache rows move to the places behind the
            prefix, the sequences get their new lengths; the rows are read back.

The tree.  The nodes of a sequence are its tokens ``starts[b]`` to
``starts[b+1]``; ``parents`` holds each one's parent as an index within the
sequence (a lower one), -1 where it follows the prefix.  In a verify call the
first node is the last token that is certain, the others are drafts.

The walk.  At a node with the target's probabilities p (logits over the
sequence's temperature; a temperature of 0 stands for the largest logit alone)
its children are tried in order, r = p at first.  Drafts drawn from q without
replacement: child x is accepted if u < r(x) / q(x), else r = (r - q)+ and q
loses x, both normalised again.  Drafts chosen without chance: accepted if
u < r(x), else r loses x.  Where no child is left the next token is drawn: the
first whose cumulative r passes the root's number.  At a temperature of 0 drafts
count as chosen: the child that is the largest logit's token is accepted.

The cache.  A page holds P tokens.  For each key/value head it holds four
arrays in turn: key codes [P][D/2], key scales [P][D/16], value codes and value
scales of the same shapes.  16 consecutive channels share a scale byte: the top
eight bits below the sign of a half-precision number d (5 exponent bits, 3
fraction bits), at most 896.  A channel is (c - 8) d for its code c in 0..15;
channel e of each eight is nibble e/2 + 4 (e%2) of their 32-bit word.
"""
import math

import torch

own = False

_DEVICE = "cuda"
_ORDER = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble of channel e of eight
_HEADS = {  # name: (query heads, key/value heads, channels)
    "64x4x192": (64, 4, 192),
    "32x8x128": (32, 8, 128),
    "16x16x64": (16, 16, 64),
    "16x2x256": (16, 2, 256),
}


def listed():
    return [
        # the smallest call: one user, a token and three drafts two of which share a parent, a short history
        dict(name="tree_small", op="tree", heads="32x8x128", seqs=1, nodes=4, length=515, window=0, page=16, act="bf16"),
        # one user's tree behind a long history that ends inside a page
        dict(name="tree_long", op="tree", heads="64x4x192", seqs=1, nodes=16, length=32765, window=0, page=64, act="bf16"),
        # 32 users' trees, ragged histories, small pages
        dict(name="tree_batch", op="tree", heads="32x8x128", seqs=32, nodes=12, length=8192, window=0, page=16, act="bf16"),
        # wide trees of a few users, as a draft model with many candidates grows them
        dict(name="tree_wide", op="tree", heads="64x4x192", seqs=8, nodes=64, length=8000, window=0, page=64, act="bf16"),
        # 16 users' trees in a sliding-window layer
        dict(name="tree_window", op="tree", heads="64x4x192", seqs=16, nodes=8, length=8000, window=512, page=64, act="bf16"),
        # the fp32 check mode
        dict(name="tree_check", op="tree", heads="16x16x64", seqs=2, nodes=7, length=999, window=0, page=32, act="f32"),
        # one user: a token and three drafts in a chain, chosen without chance
        dict(name="verify_chain", op="verify", seqs=1, nodes=4, chain=True, vocab=32768, drafts="chosen", logits="f32"),
        # a wide tree of a few users, drafts drawn from the draft head's distribution
        dict(name="verify_wide", op="verify", seqs=4, nodes=64, chain=False, vocab=32768, drafts="drawn", logits="f32"),
        # 64 users' chains with a large vocabulary, drawn drafts, bf16 logits, some users without chance
        dict(name="verify_batch", op="verify", seqs=64, nodes=4, chain=True, vocab=151936, drafts="drawn", logits="bf16"),
        # 32 users' trees with a large vocabulary, chosen drafts
        dict(name="verify_trees", op="verify", seqs=32, nodes=12, chain=False, vocab=151936, drafts="chosen", logits="f32"),
        # what one user's tree leaves in one layer's cache
        dict(name="commit_one", op="commit", heads="64x4x192", seqs=1, nodes=12, length=32765, page=64),
        # 128 users' trees, small pages
        dict(name="commit_batch", op="commit", heads="32x8x128", seqs=128, nodes=64, length=2000, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "commit"])
    if op == "verify":
        seqs = _log(rng, 1, 64)
        nodes = rng.randint(1, max(1, min(64, 384 // seqs)))
        return dict(op=op, seqs=seqs, nodes=nodes, chain=rng.choice([True, False, False]),
                    vocab=_log(rng, 1000, min(200000, 58000000 // (seqs * nodes))), drafts=rng.choice(["chosen", "drawn"]),
                    logits=rng.choice(["f32", "bf16"]))
    heads, page = rng.choice(sorted(_HEADS)), rng.choice([16, 32, 64, 128])
    if op == "commit":
        seqs, nodes = _log(rng, 1, 128), rng.randint(1, 64)
        return dict(op=op, heads=heads, seqs=seqs, nodes=nodes, length=nodes + _log(rng, 1, 250000 // seqs), page=page)
    if rng.random() < 0.15:
        nodes = rng.randint(1, 8)
        return dict(op=op, heads=heads, seqs=rng.randint(1, 4), nodes=nodes, length=nodes + _log(rng, 8, 2000), window=0, page=page, act="f32")
    seqs = _log(rng, 1, 32)
    nodes = rng.randint(1, min(64, 512 // seqs))
    return dict(op=op, heads=heads, seqs=seqs, nodes=nodes, length=nodes + _log(rng, 16, 64000 // max(seqs, nodes // 8)),
                window=rng.choice([0, 0, 512, 100]), page=page, act="bf16")


# ------------------------------------------------------------------ shapes


def _lengths(case):
    """(tokens in the cache, nodes among them) of each sequence: the first has the case's own, the others fewer."""
    n, m, lens, nodes = case.get("length", 0), case["nodes"], [], []
    for b in range(case["seqs"]):
        nodes.append(max(1, m - b * 7 % max(1, m // 3)))
        lens.append(max(nodes[-1], n - (b * 2654435761 % 1000003) * n // 2 // 1000003))
    return lens, nodes


def _hash(*v):
    h = 0
    for x in v:
        h = (h * 1000003 + x + 0x9E3779B9) * 2654435761 % (1 << 32)
        h ^= h >> 15
    return h


def _parents(case):
    """Each sequence's list of parents: the shape of a tree is the case's own (as a draft policy's is)."""
    out = []
    for b, m in enumerate(_lengths(case)[1]):
        if case.get("chain"):
            out.append(list(range(-1, m - 1)))
        else:
            out.append([-1] + [(i - 1) // 3 + _hash(b, i) % (i - (i - 1) // 3) for i in range(1, m)])
    return out


def _depths(parents):
    out = []
    for p in parents:
        out.append(out[p] + 1 if p >= 0 else 0)
    return out


def _paths(case):
    """Accepted paths, lists of nodes.  They lie behind the places they move to, as those of a wide tree do, so that a pass can be repeated."""
    out = []
    for b, m in enumerate(_lengths(case)[1]):
        k = 1 + _hash(b, 77) % 6
        rest = list(range(k, m))[:: max(1, (m - k) // max(1, k))]
        out.append([0] + rest[: k - 1])
    return out


# How often a walk goes on from a node that has children, with `prepare`'s distributions: drafts chosen without
# chance and drawn ones, in a chain and in a tree (where the branch that is taken may be a short one).
_GOES_ON = {("chosen", True): 0.70, ("chosen", False): 0.65, ("drawn", True): 0.88, ("drawn", False): 0.82}


def _rows(case):
    """Rows of logits that the walks read, on average: each one's root's and its accepted drafts'."""
    a = _GOES_ON[case["drafts"], case["chain"]]
    return sum((1 - a ** (1 + max(_depths(p)))) / (1 - a) for p in _parents(case))


def work(case):
    if case["op"] == "verify":
        v, size = case["vocab"], 4 if case["logits"] == "f32" else 2
        rows = _rows(case)
        both = 2 if case["drafts"] == "drawn" else 1
        return {"bytes": int(rows * v * size * both) + 12 * sum(_lengths(case)[1]), "flops": int(rows * v * both * 4)}
    hq, hk, d = _HEADS[case["heads"]]
    row = hk * d * 2 * 9 // 16  # a token's keys and values in the cache
    lens, nodes = _lengths(case)
    if case["op"] == "commit":
        moved = sum(len(p) for p in _paths(case))
        return {"bytes": 2 * moved * row + sum(nodes) * (row + 2 * hk * d * 2), "flops": 0}
    size, w = 2 if case["act"] == "bf16" else 4, case["window"] or 1 << 40
    pairs = seen = 0
    for n, m, parents in zip(lens, nodes, _parents(case)):
        seen += min(n, m + w - 1)
        pairs += sum(min(w, n - m + t + 1) for t in _depths(parents))
    return {"bytes": seen * row + 2 * sum(nodes) * hq * d * size, "flops": 4 * pairs * hq * d}


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


def _values(codes, scales):
    """The fp32 rows [..., D] that codes [..., D/2] and scale bytes [..., D/16] stand for."""
    b = codes.unflatten(-1, (-1, 4))
    nib = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    c = nib[..., _ORDER].flatten(-2).unflatten(-1, (-1, 16)).to(torch.float32) - 8
    d = (scales.to(torch.int16) << 7).view(torch.float16).to(torch.float32)
    return (c * d[..., None]).flatten(-2)


def _random_pages(n_pages, hk, p, d, gen):
    """Pages of random codes; scales around those that normal rows of unit variance have (0.2 to 0.5)."""
    pages = torch.randint(256, (n_pages, hk * p * d * 9 // 8), generator=gen, device=_DEVICE, dtype=torch.uint8)
    _, ks, _, vs = _arrays(pages, hk, p, d)
    for s in (ks, vs):
        s.copy_(torch.randint(100, 112, s.shape, generator=gen, device=_DEVICE, dtype=torch.uint8))
    return pages


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device=_DEVICE).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=_DEVICE)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=_DEVICE)

    lens, nodes = _lengths(case)
    starts = [0]
    for m in nodes:
        starts.append(starts[-1] + m)
    total = starts[-1]
    s = dict(case=case, starts=torch.tensor(starts, **i32), max_nodes=max(nodes))
    parents = _parents(case)
    if case["op"] != "commit":
        s["parents"] = torch.tensor([p for seq in parents for p in seq], **i32)
    if case["op"] == "verify":
        v, kind = case["vocab"], torch.float32 if case["logits"] == "f32" else torch.bfloat16
        # logits as a trained head gives them: a few likely tokens over a broad rest
        x = normal(total, v) * 2
        x.scatter_add_(1, torch.randint(v, (total, 8), generator=gen, device=_DEVICE), 10 + 2.5 * normal(total, 8))
        # a draft head's, close to them
        y = x + 0.5 * normal(total, v)
        s["logits"] = x.to(kind)
        temperature = 0.6 + 0.6 * torch.rand(case["seqs"], generator=gen, device=_DEVICE)
        temperature[5::7] = 0  # users who take the most probable token
        s["temperature"] = temperature
        y = y.to(kind)
        order = y.float()
        if case["drafts"] == "drawn":
            s["draft_logits"] = y
            # the children of a node are drawn without replacement: the largest of the log probabilities and Gumbel numbers
            t = temperature.repeat_interleave(torch.tensor(nodes, device=_DEVICE))[:, None]
            noise = -torch.log(-torch.log(torch.rand(total, v, generator=gen, device=_DEVICE).clamp(1e-20, 1 - 6e-8)))
            order = torch.where(t > 0, order / t + noise, order)
        rank, source = [0] * total, [0] * total
        for b, seq in enumerate(parents):
            had = {}
            for i, p in enumerate(seq):
                rank[starts[b] + i], source[starts[b] + i] = had.get(p, 0), starts[b] + max(p, 0)
                had[p] = had.get(p, 0) + 1
        best = order.topk(min(v, max(rank) + 1), 1).indices
        s["tokens"] = best[torch.tensor(source, device=_DEVICE), torch.tensor(rank, device=_DEVICE)].to(torch.int32)
        s["uniforms"] = torch.rand(total, generator=gen, device=_DEVICE)
        # how far the drafts go is a draft policy's own: a user's program knows it
        s["levels"] = max(max(_depths(seq)) for seq in parents)
        s["siblings"] = max(rank) + 1
        return s
    hq, hk, d = _HEADS[case["heads"]]
    page = case["page"]
    tables = [-(-n // page) for n in lens]
    n_pages = sum(tables) + 2
    s["pages"] = _random_pages(n_pages, hk, page, d, gen)
    order = torch.randperm(n_pages, generator=gen, device=_DEVICE).to(torch.int32).cpu()
    table = torch.zeros(len(lens), max(tables), dtype=torch.int32)
    used = 0
    for b, n in enumerate(tables):
        table[b, :n] = order[used:used + n]
        used += n
    s["table"] = table.to(_DEVICE)
    s["lens"] = torch.tensor(lens, **i32)
    s["max_len"] = max(lens)
    act = "f32" if case.get("act") == "f32" else "bf16"
    if case["op"] == "tree":
        s["q"] = (normal(total, hq, d) * 1.5).to(torch.float32 if act == "f32" else torch.bfloat16)
    else:
        path = torch.full((len(lens), max(nodes)), -1, dtype=torch.int32)
        for b, p in enumerate(_paths(case)):
            path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        s["path"] = path.to(_DEVICE)
        slots = [int(table[b, j // page]) * page + j % page for b, (n, m) in enumerate(zip(lens, nodes)) for j in range(n - m, n)]
        s["slots"] = torch.tensor(slots, dtype=torch.int64, device=_DEVICE)
    if own:
        import block_quantized_moe_layer_gb300 as pkg
        s["attention"] = pkg.Attention(hq, hk, d, page, n_pages, total, len(lens), max(lens), rot_dim=0,
                                       act=pkg.ACT_F32 if act == "f32" else pkg.ACT_BF16, window=case.get("window", 0))
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return {"tree": _tree, "verify": _verify, "commit": _commit}[s["case"]["op"]](s)


def _padded(s):
    """(node of each place [sequence, place], whether there is one)."""
    nodes = s["starts"][1:] - s["starts"][:-1]
    at = torch.arange(s["max_nodes"], device=_DEVICE)
    there = at < nodes[:, None]
    return (s["starts"][:-1, None] + at).clamp(max=int(s["parents"].shape[0]) - 1).long(), there


def _tree(s):
    case = s["case"]
    if own:
        return s["attention"].forward(s["q"], s["pages"], s["starts"], s["lens"], s["table"], s["max_nodes"], s["max_len"],
                                      parents=s["parents"])
    hq, hk, d = _HEADS[case["heads"]]
    p, g = case["page"], hq // hk
    n = -(-s["max_len"] // p)

    def rows(codes, scales):  # [sequence, head, token, channel] of the sequences' pages in order
        pick = s["table"][:, :n].long()
        return _values(codes[pick], scales[pick]).permute(0, 2, 1, 3, 4).flatten(2, 3)

    kc, ks, vc, vs = _arrays(s["pages"], hk, p, d)
    at, there = _padded(s)
    m = s["max_nodes"]
    # ancestors: a node's own, its parent's, and so on up
    up = torch.where(there, s["parents"][at], -1).long()
    anc = torch.zeros(*at.shape, m, dtype=torch.bool, device=_DEVICE)
    here = torch.arange(m, device=_DEVICE).expand_as(up)
    for _ in range(m):
        anc |= (here[..., None] == torch.arange(m, device=_DEVICE)) & (here >= 0)[..., None]
        here = torch.where(here >= 0, up.gather(1, here.clamp(min=0)), -1)
    depth = anc.sum(-1) - 1
    first = s["lens"] - (s["starts"][1:] - s["starts"][:-1])
    key = torch.arange(n * p, device=_DEVICE)
    where = first[:, None] + depth
    sees = (key < first[:, None, None]).expand(-1, m, -1)
    node = (key - first[:, None]).clamp(0, m - 1)[:, None].expand(-1, m, -1)
    inside = ((key >= first[:, None]) & (key < s["lens"][:, None]))[:, None]
    sees = sees | (inside & anc.gather(2, node))
    if case["window"]:
        position = torch.where(inside, first[:, None, None] + depth.gather(1, node[:, 0]).unsqueeze(1), key)
        sees = sees & (position > where[..., None] - case["window"])
    q = s["q"][at].to(torch.float32).unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = q @ rows(kc, ks).transpose(2, 3) * d ** -0.5
    sees = sees[:, None].repeat(1, 1, g, 1)
    scores = scores.masked_fill_(~sees, -math.inf)
    most = scores.amax(-1, keepdim=True)
    scores = (scores - torch.where(most > -math.inf, most, 0.0)).exp_()
    out = (scores @ rows(vc, vs)) / scores.sum(-1, keepdim=True)
    out = out.unflatten(2, (g, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return out[there].to(s["q"].dtype)


def _verify(s):
    drawn = s["case"]["drafts"] == "drawn"
    if own:
        import block_quantized_moe_layer_gb300 as pkg
        r = pkg.verify_sample(s["logits"], s["tokens"], s["parents"], s["starts"], s["uniforms"], s["max_nodes"],
                              draft_logits=s.get("draft_logits"), temperature=s["temperature"])
        return [r["path"], r["n_accepted"], r["next"]]
    at, there = _padded(s)
    n_seqs, m = at.shape
    up = torch.where(there, s["parents"][at], -1)
    tokens, uniforms = s["tokens"][at].long(), s["uniforms"][at].double()
    greedy = (s["temperature"] == 0)[:, None]
    t = torch.where(greedy, 1.0, s["temperature"].double()[:, None])

    def probabilities(logits, node):
        x = logits[node].double()
        # 64 bits: a number next to the border of two tokens takes the right one
        e = ((x - x.amax(1, keepdim=True)) / t).exp()
        first = torch.where(x == x.amax(1, keepdim=True), torch.arange(x.shape[1], device=_DEVICE), x.shape[1]).amin(1, keepdim=True)
        one = torch.zeros_like(e).scatter_(1, first, 1.0)
        return torch.where(greedy, one, e / e.sum(1, keepdim=True))

    b = torch.arange(n_seqs, device=_DEVICE)
    node = torch.zeros(n_seqs, dtype=torch.int64, device=_DEVICE)
    path = torch.full((n_seqs, m), -1, dtype=torch.int32, device=_DEVICE)
    path[:, 0] = 0
    walking = torch.ones(n_seqs, dtype=torch.bool, device=_DEVICE)
    r = None
    for level in range(s["levels"] + 1):
        p = probabilities(s["logits"], at[b, node])
        r = p if r is None else torch.where(walking[:, None], p, r)
        # the children of the node each sequence stands at, in order; m: no more
        child = torch.where(there & (up == node[:, None]), torch.arange(m, device=_DEVICE), m).sort(1).values
        q = left = None
        if drawn:
            q = probabilities(s["draft_logits"], at[b, node])
            left = torch.ones(n_seqs, 1, dtype=torch.float64, device=_DEVICE)  # of q
        open_ = walking
        walking = torch.zeros_like(walking)
        for k in range(min(s["siblings"], m)):
            c = child[:, k].clamp(max=m - 1)
            tries = open_ & (child[:, k] < m)
            x = tokens[b, c][:, None]
            total = r.sum(1, keepdim=True)
            mine = r.gather(1, x)
            wins = uniforms[b, c][:, None] * total < mine
            rest = r.scatter(1, x, 0.0)
            if drawn:
                qx = q.gather(1, x)
                wins = torch.where(greedy, wins, uniforms[b, c][:, None] * total * qx < mine * left)
                rest = torch.where(greedy, rest, (r - q * (total / left)).clamp(min=0))
                left = torch.where(tries[:, None] & ~wins, left - qx, left)
            wins = wins[:, 0] & tries
            r = torch.where((tries & ~wins)[:, None], rest, r)
            if level + 1 < m:
                path[:, level + 1] = torch.where(wins, c.to(torch.int32), path[:, level + 1])
            node = torch.where(wins, c, node)
            walking |= wins
            open_ = open_ & ~wins
    mass = r.cumsum(1)
    nxt = (mass <= uniforms[:, :1] * mass[:, -1:]).sum(1).clamp(max=r.shape[1] - 1)
    return [path, (path >= 0).sum(1).to(torch.int32) - 1, nxt.to(torch.int32)]


def _commit(s):
    case = s["case"]
    if own:
        lens = s["attention"].commit(s["pages"], s["starts"], s["lens"], s["table"], s["path"], s["max_len"])
        keys, values = s["attention"].read(s["slots"], s["pages"])
        return [lens, keys, values]
    hq, hk, d = _HEADS[case["heads"]]
    p = case["page"]
    first = (s["lens"] - (s["starts"][1:] - s["starts"][:-1])).long()[:, None]
    taken = s["path"] >= 0
    b = torch.arange(len(first), device=_DEVICE)[:, None]

    def slots(at):
        return s["table"][b, at // p].long() * p + at % p

    src = slots(first + torch.where(taken, s["path"].long(), 0))[taken]
    dst = slots((first + torch.arange(s["max_nodes"], device=_DEVICE)).minimum(s["lens"].long()[:, None] - 1))[taken]
    read = []
    for a in _arrays(s["pages"], hk, p, d):
        a[dst // p, :, dst % p] = a[src // p, :, src % p]
        read.append(a[s["slots"] // p, :, s["slots"] % p])
    lens = (first[:, 0] + taken.sum(1)).to(torch.int32)
    return [lens, _values(*read[:2]).to(torch.bfloat16), _values(*read[2:]).to(torch.bfloat16)]


# ------------------------------------------------------------------ from the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "commit": _exact_commit}[case["op"]](s)


def _cached(s, b, h, n):
    """Keys and values [n, D] of one head of a sequence, word by word."""
    _, hk, d = _HEADS[s["case"]["heads"]]
    p = s["case"]["page"]
    mine = s["pages"].view(-1, hk, p * d * 9 // 8)[s["table"][b, :-(-n // p)].long(), h]
    both = []
    for at in (0, p * d * 9 // 16):
        words = mine[:, at:at + p * d // 2].contiguous().view(torch.int32)
        scales = mine[:, at + p * d // 2:at + p * d * 9 // 16].long().reshape(-1, d // 16)[:n]
        codes = torch.stack([(words >> (4 * (e // 2 + 4 * (e % 2)))) & 15 for e in range(8)], -1).reshape(-1, d)[:n]
        e, f = scales // 8, (scales % 8).double()
        step = torch.where(e > 0, (8 + f) * torch.exp2((e - 18).double()), f * 2.0 ** -17)
        both.append((codes.double() - 8) * step.repeat_interleave(16, 1))
    return both


def _exact_tree(s):
    hq, hk, d = _HEADS[s["case"]["heads"]]
    g, w = hq // hk, s["case"]["window"] or 1 << 40
    q = s["q"].double()
    out = torch.zeros_like(q)
    starts = s["starts"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        a, e = starts[b], starts[b + 1]
        parents, first = s["parents"][a:e].tolist(), n - (e - a)
        hidden = torch.ones(e - a, n, dtype=torch.bool)
        for i in range(e - a):
            line = []  # the node and its ancestors, upwards
            j = i
            while j >= 0:
                line.append(first + j)
                j = parents[j]
            line = (line + list(range(first - 1, -1, -1)))[:w]
            hidden[i, line] = False
        hidden = hidden.to(q.device)
        for h in range(hk):
            keys, values = _cached(s, b, h, n)
            for i in range(h * g, (h + 1) * g):
                z = (q[a:e, i] @ keys.T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                out[a:e, i] = torch.softmax(z, 1) @ values
    return out


def _exact_verify(s):
    starts, paths, nexts = s["starts"].tolist(), [], []
    tokens, uniforms, temperature = s["tokens"].tolist(), s["uniforms"].tolist(), s["temperature"].tolist()
    for b in range(len(starts) - 1):
        a, e = starts[b], starts[b + 1]
        parents = s["parents"][a:e].tolist()

        def softmax(x):
            if temperature[b] > 0:
                return torch.softmax(x.double() / temperature[b], 0)
            one = torch.zeros_like(x, dtype=torch.float64)
            one[int(torch.nonzero(x == x.max())[0])] = 1
            return one

        line, at = [0], 0
        while at is not None:
            r = softmax(s["logits"][a + at])
            q = softmax(s["draft_logits"][a + at]) if "draft_logits" in s and temperature[b] > 0 else None
            here, at = at, None
            for c in range(here + 1, e - a):
                if parents[c] != here:
                    continue
                x, u = tokens[a + c], uniforms[a + c]
                if float(r[x]) > u * (1.0 if q is None else float(q[x])):
                    line.append(c)
                    at = c
                    break
                if q is None:
                    r[x] = 0
                else:
                    r = (r - q).clamp(min=0)
                    q[x] = 0
                    q = q / q.sum()
                if float(r.sum()) > 0:
                    r = r / r.sum()
        mass = r.cumsum(0)
        nexts.append(int(torch.searchsorted(mass, uniforms[a] * mass[-1:], right=True)[0].clamp(max=len(r) - 1)))
        paths.append(line + [-1] * (s["max_nodes"] - len(line)))
    i32 = dict(dtype=torch.int32, device=s["logits"].device)
    return [torch.tensor(paths, **i32), torch.tensor([sum(c >= 0 for c in p) - 1 for p in paths], **i32), torch.tensor(nexts, **i32)]


def _exact_commit(s):
    _, hk, _ = _HEADS[s["case"]["heads"]]
    starts, lens, keys, values = s["starts"].tolist(), [], [], []
    for b, n in enumerate(s["lens"].tolist()):
        m = starts[b + 1] - starts[b]
        path = [c for c in s["path"][b].tolist() if c >= 0]
        lens.append(n - m + len(path))
        rows = path + list(range(len(path), m))
        both = [_cached(s, b, h, n) for h in range(hk)]
        keys.append(torch.stack([k[n - m:][rows] for k, _ in both], 1))
        values.append(torch.stack([v[n - m:][rows] for _, v in both], 1))
    return [torch.tensor(lens, dtype=torch.int32, device=s["lens"].device), torch.cat(keys), torch.cat(values)]
