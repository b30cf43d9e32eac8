"""Sampled verification of draft trees against the fp64 oracle.

Paths and tokens are whole numbers: equal.  Weights are right to 2^-32 (a
residual's error grows with what is taken out), so a number that lies within
2^-26 of the border between two outcomes, which the oracle reports, may go
either way; among these inputs that is 1 in 10^4 at most.
"""
import numpy as np
import pytest
import torch

import block_quantized_moe_layer_gb300 as pkg
from oracle import tree as ot

pytestmark = pytest.mark.gpu

NEAR = 2.0 ** -26


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _tree(rng, m, chain=False):
    return list(range(-1, m - 1)) if chain else [-1][:m] + [int(rng.integers(max(0, (i - 1) // 3), i)) for i in range(1, m)]


def _peaked(rng, n, V, scale=2.0):
    x = rng.normal(size=(n, V)) * scale
    for r in x:
        r[rng.integers(0, V, 4)] += rng.normal(size=4) * 2 + np.log(V)
    return x


def _case(rng, V, sizes, drawn, dtype, chain=False, temperature=None, replacement=False, pad=0, offset=0, logits=None, draft=None,
          tokens=None, uniforms=None, trees=None, max_nodes=None):
    trees = [_tree(rng, m, chain) for m in sizes] if trees is None else trees
    N = sum(sizes)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    x = _peaked(rng, N, V) if logits is None else logits
    y = x + 0.5 * rng.normal(size=x.shape) if draft is None else draft
    full = torch.zeros(max(N, 1), V + pad + offset, dtype=dtype, device="cuda")

    def put(a):
        t = full.clone()[:N, offset:offset + V]
        t.copy_(torch.tensor(np.asarray(a), device="cuda"))
        return t

    x, y = put(x), put(y)
    xs, ys = x.double().cpu().numpy(), y.double().cpu().numpy()
    temperature = np.ones(len(sizes), np.float32) if temperature is None else np.asarray(temperature, np.float32)
    if tokens is None:
        tokens = np.zeros(N, np.int64)
        for b, t in enumerate(trees):
            used = {}
            for i, p in enumerate(t):
                if not 0 <= p < i:
                    continue
                q = ot.distribution(ys[starts[b] + p], max(float(temperature[b]), 0.05) if 0 <= temperature[b] <= 1e6 else 1.0)
                k = used.setdefault(p, [])
                if drawn and replacement:
                    tokens[starts[b] + i] = rng.choice(V, p=q)
                else:
                    q = q.copy()
                    q[k] = 0
                    free = np.flatnonzero(q > 0)
                    tokens[starts[b] + i] = (-1 if len(free) == 0 else rng.choice(V, p=q / q.sum()) if drawn else int(np.argmax(q)))
                    if tokens[starts[b] + i] >= 0:
                        k.append(tokens[starts[b] + i])
    u = rng.random(N).astype(np.float32).clip(max=np.float32(1 - 2.0 ** -24)) if uniforms is None else np.asarray(uniforms, np.float32)
    width = max(max(sizes), 1) if max_nodes is None else max_nodes
    args = (x, _i32(tokens), None if chain else _i32([p for t in trees for p in t]), _i32(starts), torch.tensor(u, device="cuda"), width)
    kw = dict(draft_logits=y if drawn else None, temperature=torch.tensor(temperature, device="cuda"), replacement=replacement)
    r = pkg.verify_sample(*args, **kw)
    again = pkg.verify_sample(*args, **kw)
    assert all(torch.equal(r[k], again[k]) for k in r)
    path, acc, nxt = (r[k].cpu().numpy() for k in ("path", "n_accepted", "next"))
    compared = 0
    for b, m in enumerate(sizes):
        if m == 0:
            assert acc[b] == -1 and nxt[b] == -1 and (path[b] == -1).all()
            continue
        sl = slice(starts[b], starts[b] + min(m, width))
        want, token, gap = ot.verify(xs[sl], tokens[sl], trees[b][:width], u[sl].astype(np.float64), ys[sl] if drawn else None,
                                     float(temperature[b]), replacement)
        if gap < NEAR:
            continue
        compared += 1
        assert path[b, :len(want)].tolist() == want and (path[b, len(want):] == -1).all(), (b, path[b], want)
        assert acc[b] == len(want) - 1 and nxt[b] == token, (b, nxt[b], token, want)
    assert compared >= 0.98 * sum(m > 0 for m in sizes) - 1
    return path, acc, nxt


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 100, 1000, 4099, 33001])
def test_trees_and_chains(V, drawn, dtype):
    rng = np.random.default_rng(V + drawn)
    few = V > 5000
    for chain in (True, False):
        sizes = [4, 1, 12, 3] if few else [4, 1, 12, 3, 0, 7, 30, 64, 2, 5]
        _case(rng, V, sizes, drawn, dtype, chain, temperature=0.5 + rng.random(len(sizes)))


@pytest.mark.parametrize("V,n_seqs", [(40000, 1), (151936, 2), (9000, 40), (2100, 200)])
def test_cluster_sizes(V, n_seqs):
    rng = np.random.default_rng(V)
    for drawn in (False, True):
        _case(rng, V, [3] * n_seqs, drawn, torch.float32)


@pytest.mark.parametrize("V,dtype", [(300001, torch.float32), (100003, torch.bfloat16), (20011, torch.float32)])
def test_many_sequences_of_long_rows(V, dtype):
    """One block a sequence, so that a thread has many vectors of the range that holds the next token (most sequences are empty here)."""
    rng = np.random.default_rng(V)
    sizes = [0] * 160
    for b in range(0, 160, 20):
        sizes[b] = 2 + b // 20 % 3
    for drawn in (False, True):
        _case(rng, V, sizes, drawn, dtype, temperature=np.linspace(0.5, 1.5, 160))


def test_independent_draws():
    rng = np.random.default_rng(21)
    for V in (3, 50, 2000):
        _case(rng, V, [9] * 20, True, torch.float32, replacement=True, trees=[[-1] + [0] * 8] * 20)
        _case(rng, V, [9] * 20, True, torch.bfloat16, replacement=True)


def test_many_siblings():
    rng = np.random.default_rng(22)
    for drawn in (False, True):
        x = rng.normal(size=(64 * 6, 500))
        _case(rng, 500, [64] * 6, drawn, torch.float32, trees=[[-1] + [0] * 63] * 6, logits=x, draft=x + rng.normal(size=x.shape))


def test_temperatures():
    rng = np.random.default_rng(23)
    t = [0.0, 1e-7, 1e-6, 0.01, 0.3, 1.0, 5.0, 1e4, 1e6, -1.0, float("nan"), float("inf"), 2e6]
    for drawn in (False, True):
        for dtype in (torch.float32, torch.bfloat16):
            _, acc, nxt = _case(rng, 777, [6] * len(t), drawn, dtype, temperature=t)
            assert (nxt[9:] == -1).all() and (acc[9:] == 0).all()
    # without temperatures: 1
    x = torch.randn(4, 50, device="cuda")
    args = (x, _i32([0, 1, 2, 3]), None, _i32([0, 4]), torch.rand(4, device="cuda"), 4)
    a, b = pkg.verify_sample(*args), pkg.verify_sample(*args, temperature=torch.ones(1, device="cuda"))
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_greedy_is_verify_accept():
    rng = np.random.default_rng(24)
    for _ in range(20):
        k, V = int(rng.integers(0, 8)), int(rng.integers(2, 3000))
        logits = torch.tensor(rng.integers(0, 30, (k + 1, V)), dtype=torch.float32, device="cuda")
        draft = logits[:k].argmax(1).to(torch.int32)
        if k > 2:
            draft[k - 1] = (draft[k - 1] + 1) % V
        want = pkg.verify_accept(draft, logits).tolist()
        tokens = torch.cat([draft.new_zeros(1), draft])
        r = pkg.verify_sample(logits, tokens, None, _i32([0, k + 1]), torch.rand(k + 1, device="cuda"), k + 1,
                              temperature=torch.zeros(1, device="cuda"))
        assert [int(r["n_accepted"]), int(r["next"])] == want


def test_masks_and_odd_rows():
    """Masked logits, whole rows of them, NaN and infinities, absent and repeated drafts, bad parents."""
    rng = np.random.default_rng(25)
    V, low = 600, float(torch.finfo(torch.float32).min)
    for drawn in (False, True):
        for dtype, mask in ((torch.float32, -np.inf), (torch.float32, low), (torch.bfloat16, -np.inf)):
            sizes = [5] * 24
            x = _peaked(rng, 120, V)
            x[:, rng.random(V) < 0.9] = mask
            y = x + 0.3 * rng.normal(size=x.shape) if mask == -np.inf else np.where(x == low, low, x + 0.3 * rng.normal(size=x.shape))
            keep = np.flatnonzero(x[0] > -1e30)
            x[5 * 3] = -np.inf
            x[5 * 4, 7] = np.nan
            x[5 * 5, 7] = np.inf
            x[5 * 6] = mask
            x[5 * 6, keep[0]] = 1.0  # one token is left
            y[5 * 6] = x[5 * 6]
            y[5 * 7] = -np.inf  # a draft row without a distribution
            y[5 * 8, 3] = np.nan
            tokens = keep[rng.integers(0, len(keep), 120)]
            tokens[5 * 9 + 1:5 * 9 + 5] = [-1, V, 2 ** 31 - 1, -2 ** 31]
            tokens[5 * 10 + 1:5 * 10 + 5] = keep[0]
            trees = [_tree(rng, 5) for _ in sizes]
            trees[10] = [-1, 0, 0, 0, 0]
            trees[11] = [3, -1, 2, 7, 3]
            trees[12] = [-1, 0, 5, -2, 1]
            _case(rng, V, sizes, drawn, dtype, logits=x, draft=y, tokens=tokens, trees=trees)


def test_offset_logits():
    """Large common offsets cost nothing of the differences that are left."""
    rng = np.random.default_rng(26)
    for offset in (-3.0e5, 1.0e4, 3.0e7):
        x = np.round(_peaked(rng, 60, 300) * 4) * (1 if abs(offset) < 1e6 else 4) + offset
        _case(rng, 300, [5] * 12, False, torch.float32, logits=x, temperature=[2.0] * 12)
        _case(rng, 300, [5] * 12, True, torch.float32, logits=x, draft=x + np.round(rng.normal(size=x.shape)) * 4, temperature=[2.0] * 12)


def test_strides_and_alignment():
    rng = np.random.default_rng(27)
    for pad, offset in ((1, 0), (3, 1), (8, 3), (5, 2)):
        for dtype in (torch.float32, torch.bfloat16):
            for V in (37, 2049):
                _case(rng, V, [4, 6, 2], True, dtype, pad=pad, offset=offset)


def test_numbers_at_the_ends():
    """Numbers of 0 and of 1 - 2^-24, equal logits, drafts equal to the target."""
    rng = np.random.default_rng(28)
    one = 1 - 2.0 ** -24
    for V in (1, 5, 3000):
        x = np.zeros((40, V))
        path, acc, nxt = _case(rng, V, [4] * 10, False, torch.float32, logits=x, uniforms=[0.0] * 40, chain=True)
        assert (acc == 3).all() and (nxt == 0).all()
        _case(rng, V, [4] * 10, True, torch.float32, logits=x, draft=x, uniforms=[one] * 40, chain=True)
        x = torch.zeros(1, V, device="cuda")
        r = pkg.verify_sample(x, _i32([0]), None, _i32([0, 1]), torch.tensor([one], device="cuda"), 1)
        assert int(r["next"]) == V - 1


def test_drafts_nearly_the_target():
    """Draft distributions that are the target's but for a few tokens, and scaled or far ones: what is left of the target
    is a few tokens, or nearly all."""
    rng = np.random.default_rng(31)
    for V in (300, 20000):
        x = _peaked(rng, 60, V)
        swapped = x.copy()
        order = np.argsort(-x, 1)
        rows = np.arange(60)
        for a, b in ((0, 3), (1, 40), (2, 100)):
            swapped[rows, order[:, a]], swapped[rows, order[:, b]] = x[rows, order[:, b]], x[rows, order[:, a]]
        for y in (swapped, x + 5.0, x + 1e-4 * rng.normal(size=x.shape), 0.3 * x, 3 * x, rng.normal(size=x.shape), np.roll(x, 1, 1)):
            for top in (3, 40):  # drafts that the draft head likes, or the target hardly
                best = np.argsort(-y, 1)[:, :top]
                tokens = np.array([best[5 * (i // 5) + max(0, i % 5 - 1), (i % 5 * 7) % top] for i in range(60)])
                for replacement in (False, True):
                    _case(rng, V, [5] * 12, True, torch.float32, logits=x, draft=y, tokens=tokens, replacement=replacement,
                          trees=[[-1, 0, 0, 1, 2]] * 6 + [[-1, 0, 1, 2, 3]] * 6)


def test_more_nodes_than_said():
    rng = np.random.default_rng(29)
    _case(rng, 200, [10, 3, 8], True, torch.float32, max_nodes=5)


def test_starts_out_of_range():
    x = torch.randn(6, 20, device="cuda")
    args = (x, _i32([0] * 6), _i32([-1, 0, 1, -1, 0, 1]))
    r = pkg.verify_sample(*args, _i32([0, 3, 3, 7]), torch.rand(6, device="cuda"), 4)
    assert r["n_accepted"].tolist()[1:] == [-1, -1] and r["next"].tolist()[1:] == [-1, -1] and (r["path"][1:] == -1).all()
    assert r["n_accepted"][0] >= 0 and r["next"][0] >= 0
    r = pkg.verify_sample(*args, _i32([-1, 3, 2]), torch.rand(6, device="cuda"), 4)
    assert r["next"].tolist() == [-1, -1]
    r = pkg.verify_sample(*args, _i32([0]), torch.rand(6, device="cuda"), 4)
    assert r["path"].shape == (0, 4)


@pytest.mark.parametrize("mode", ["chosen", "drawn", "independent"])
def test_tokens_are_distributed_as_the_target(mode):
    """The token after the root, over many sequences: each frequency within 5 standard deviations of p."""
    n, V = 40000, 6
    g = torch.Generator(device="cuda").manual_seed(5)
    p = torch.tensor([2.0, 1.0, 0.5, 0.0, -1.0, 0.3], device="cuda")
    q = torch.tensor([0.0, 1.5, 0.5, 1.0, 0.5, -0.5], device="cuda")
    pq = torch.softmax(q.double(), 0).expand(n, V)
    if mode == "chosen":
        kids = torch.tensor([1, 3], device="cuda").expand(n, 2)
    else:
        kids = torch.multinomial(pq, 2, replacement=mode == "independent", generator=g)
    tokens = torch.cat([torch.zeros(n, 1, device="cuda"), kids], 1).to(torch.int32).reshape(-1)
    r = pkg.verify_sample(p.expand(3 * n, V).contiguous(), tokens, _i32([-1, 0, 0]).repeat(n),
                          torch.arange(0, 3 * n + 1, 3, dtype=torch.int32, device="cuda"),
                          torch.rand(3 * n, generator=g, device="cuda"), 3,
                          draft_logits=None if mode == "chosen" else q.expand(3 * n, V).contiguous(), replacement=mode == "independent")
    took = r["path"][:, 1].long()
    first = torch.where(took > 0, tokens.view(n, 3).gather(1, took.clamp(min=0)[:, None])[:, 0].long(), r["next"].long())
    share = torch.bincount(first, minlength=V).double() / n
    want = torch.softmax(p.double(), 0)
    assert ((share - want).abs() <= 5 * (want * (1 - want) / n).sqrt()).all(), (share, want)


def test_stream_and_capture():
    rng = np.random.default_rng(30)
    x = torch.tensor(_peaked(rng, 8, 5000), dtype=torch.float32, device="cuda")
    u, tokens = torch.rand(8, device="cuda"), x.argmax(1).to(torch.int32).roll(1)
    args = (x, tokens, None, _i32([0, 4, 8]), u, 4)
    want = pkg.verify_sample(*args)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = pkg.verify_sample(*args, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = pkg.verify_sample(*args)
    for _ in range(5):
        u.copy_(torch.rand(8, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        want = pkg.verify_sample(*args)
        assert all(torch.equal(want[k], r[k]) for k in want)


def test_refusals():
    x = torch.randn(4, 20, device="cuda")
    tokens, starts, u = _i32([0] * 4), _i32([0, 4]), torch.rand(4, device="cuda")
    good = dict(logits=x, tokens=tokens, parents=None, starts=starts, uniforms=u, max_nodes=4)
    for change, what in ((dict(logits=x.double()), "logits"), (dict(logits=x[0]), "logits"), (dict(logits=x.t()), "contiguous"),
                         (dict(logits=x.cpu()), "logits"), (dict(tokens=tokens.long()), "tokens"), (dict(tokens=tokens[:3]), "tokens"),
                         (dict(parents=tokens[:3]), "parents"), (dict(uniforms=u.double()), "uniforms"), (dict(uniforms=u.cpu()), "uniforms"),
                         (dict(starts=starts.long()), "starts"), (dict(max_nodes=0), "max_nodes"), (dict(max_nodes=65), "max_nodes"),
                         (dict(draft_logits=x.to(torch.bfloat16)), "draft_logits"), (dict(draft_logits=x[:3]), "draft_logits"),
                         (dict(temperature=torch.ones(2, device="cuda")), "temperature"),
                         (dict(temperature=torch.ones(1, device="cuda").double()), "temperature"),
                         (dict(logits=x[:1].expand(4, 20)), "stride")):
        with pytest.raises(pkg.MoEError, match=what):
            pkg.verify_sample(**{**good, **change})
