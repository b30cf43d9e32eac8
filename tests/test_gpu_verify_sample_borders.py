"""Sampled verification with numbers beside the border of two outcomes, and odd rows shared by many blocks.

A probability or a sum of them is right to 2^-32 of the row's sum.  A token's
border, and a chosen draft's, is one such number, so a uniform number 2^-31 from
it falls on its own side; a drawn draft's is u = p(x) / q(x) <= 1, two of them:
2^-30.  (Borders are computed in numpy's long double; the uniform numbers are
whole fp32 numbers.)
"""
import numpy as np
import pytest
import torch

import block_quantized_moe_layer_gb300 as pkg
from tests.test_gpu_verify_sample import _case, _i32, _peaked, _tree

pytestmark = pytest.mark.gpu


def _weights(x, temperature):
    """Probabilities of a row in long double."""
    x = np.asarray(x, np.longdouble) / np.longdouble(np.float32(temperature))
    e = np.exp(x - x.max())
    return e / e.sum()


def _beside(borders, near):
    """fp32 numbers u whose nearest border (of ascending ones) is between near and 2 near away."""
    mid = borders.astype(np.float32)
    u = np.unique(np.concatenate([np.nextafter(mid, np.float32(0)), mid, np.nextafter(mid, np.float32(1))]))
    u = u[(u >= 0) & (u < 1)]
    at = np.searchsorted(borders, u.astype(np.longdouble))
    far = np.concatenate([[-np.inf], borders, [np.inf]]).astype(np.longdouble)
    d = np.minimum(u - far[at], far[at + 1] - u)
    return u[(d >= near) & (d <= 2 * near)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n_seqs", [(3000, 2), (33001, 1), (151936, 2), (151936, 40), (300001, 160)])
def test_tokens_beside_their_borders(V, n_seqs, dtype):
    """Draws of the next token: one row for all the sequences of a call, `n_seqs` with nodes at a time."""
    rng = np.random.default_rng(V + n_seqs)
    row = torch.tensor(_peaked(rng, 1, V), dtype=torch.float32).to(dtype)
    for temperature in (1.0, 0.7):
        w = _weights(row.double().numpy()[0], temperature)
        mass = np.cumsum(w)
        places = _beside(mass, 2.0 ** -31)
        assert len(places) >= 8
        rng.shuffle(places)
        places = places[:max(2 * n_seqs, 16)]
        logits = row.cuda().expand(n_seqs, V).contiguous()
        t = torch.full((n_seqs,), temperature, device="cuda")
        for at in range(0, len(places), n_seqs):
            part = np.resize(places[at:at + n_seqs], n_seqs)
            u = torch.tensor(part, device="cuda")
            r = pkg.verify_sample(logits, _i32([0] * n_seqs), None, _i32(range(n_seqs + 1)), u, 1, temperature=t)
            # the first token whose cumulative mass passes the number
            want = np.searchsorted(mass, part.astype(np.longdouble) * mass[-1], side="right")
            assert r["next"].tolist() == want.tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("V", [40, 20011])
def test_drafts_beside_their_borders(V, drawn, dtype):
    """A draft's number on either side of its border."""
    rng = np.random.default_rng(V + drawn)
    n = 16 if V > 1000 else 64
    x, y, tokens, numbers, want = [], [], [], [], []
    near = 2.0 ** -30 if drawn else 2.0 ** -31
    while len(want) < n:
        a = rng.normal(size=V) * 2
        top = int(rng.integers(V))
        a[top] = np.log(np.exp(a).sum()) + rng.normal()
        b = a + 0.3 * rng.normal(size=V)
        if drawn:
            b[top] += 0.7
        a, b = (torch.tensor(v, dtype=torch.float32).to(dtype).double().numpy() for v in (a, b))
        p, q = _weights(a, 1.0)[top], _weights(b, 1.0)[top]
        for u in _beside(np.array([p / q if drawn else p]), near)[:1]:
            x += [a, a]
            y += [b, b]
            tokens += [0, top]
            numbers += [0.5, float(u)]
            want.append(1 if np.longdouble(u) * (q if drawn else 1) < p else 0)
    rows, drafts = (torch.tensor(np.array(v), dtype=torch.float32, device="cuda").to(dtype) for v in (x, y))
    r = pkg.verify_sample(rows, _i32(tokens), None, _i32(range(0, 2 * n + 1, 2)), torch.tensor(numbers, dtype=torch.float32, device="cuda"), 2,
                          draft_logits=drafts if drawn else None)
    assert r["n_accepted"].tolist() == want and 0 < sum(want) < n


V16 = 20000  # a row that 16 blocks share where a call has few sequences


@pytest.mark.parametrize("drawn", [False, True])
def test_temperatures_of_shared_rows(drawn):
    rng = np.random.default_rng(41)
    t = [0.0, 1e-7, 1e-6, 0.01, 0.3, 1.0, 5.0, 1e4, 1e6, -1.0, float("nan"), float("inf"), 2e6]
    for dtype in (torch.float32, torch.bfloat16):
        _, acc, nxt = _case(rng, V16, [5] * len(t), drawn, dtype, temperature=t)
        assert (nxt[9:] == -1).all() and (acc[9:] == 0).all()


def test_greedy_ties_between_blocks():
    """The largest logit several times, in slices of different blocks: the lowest id."""
    rng = np.random.default_rng(42)
    for V in (V16, 33001, 151936):
        for dtype in (torch.float32, torch.bfloat16):
            x = torch.tensor(rng.integers(0, 30, (4, V)), dtype=torch.float32).to(dtype)
            ties = [np.sort(rng.choice(V, 5, replace=False)) for _ in range(4)]
            for i, at in enumerate(ties):
                x[i, at] = 40.0
            first = [int(at[0]) for at in ties]
            tokens = _i32([0, first[0], first[1], int(ties[2][1])])  # (the last: a tie, but not the lowest)
            r = pkg.verify_sample(x.cuda(), tokens, None, _i32([0, 4]), torch.rand(4, device="cuda"), 4, temperature=torch.zeros(1, device="cuda"))
            assert r["path"][0].tolist() == [0, 1, 2, -1] and r["next"].tolist() == [first[2]]
            assert pkg.verify_accept(tokens[1:], x.float().cuda()).tolist() == [2, first[2]]


@pytest.mark.parametrize("drawn", [False, True])
def test_masks_and_odd_rows_of_shared_rows(drawn):
    """NaN, infinities, whole masked slices and rows, one token that is left, in slices of different blocks; absent and
    repeated drafts, bad parents."""
    rng = np.random.default_rng(43)
    V, low = V16, float(torch.finfo(torch.float32).min)
    for dtype, mask in ((torch.float32, -np.inf), (torch.float32, low), (torch.bfloat16, -np.inf)):
        for at in (0, V // 2 + 1, V - 1):
            for first in range(0, 16, 4):
                sizes = [5] * 4
                x = _peaked(rng, 20, V)
                x[:, rng.random(V) < 0.9] = mask
                x[:, V // 4:V // 2] = mask  # whole slices
                x[:, at] = 0.5
                y = x + 0.3 * rng.normal(size=x.shape) if mask == -np.inf else np.where(x == low, low, x + 0.3 * rng.normal(size=x.shape))
                keep = np.flatnonzero(x[0] > -1e30)
                tokens = keep[rng.integers(0, len(keep), 20)]
                trees = [_tree(rng, 5) for _ in sizes]
                if first == 0:
                    x[0] = -np.inf
                    x[5, at] = np.nan
                    x[10, at] = np.inf
                    x[15] = mask
                    x[15, at] = 1.0  # one token is left
                    y[15] = x[15]
                elif first == 4:
                    y[0] = -np.inf  # a draft row without a distribution
                    y[5, at] = np.nan
                    tokens[11:15] = [-1, V, 2 ** 31 - 1, -2 ** 31]
                    tokens[16:20] = at
                    trees[3] = [-1, 0, 0, 0, 0]
                elif first == 8:
                    trees[0], trees[1] = [3, -1, 2, 7, 3], [-1, 0, 5, -2, 1]
                    x[10:] = mask  # a row with two tokens, in different blocks or one
                    x[10:, [at, V // 3]] = [1.0, 0.3]
                    y[10:] = x[10:]
                    tokens[10:] = [at, V // 3] * 5
                _, acc, nxt = _case(rng, V, sizes, drawn, dtype, logits=x, draft=y, tokens=tokens, trees=trees)
                if first == 0:
                    assert (nxt[:3] == -1).all() and (acc[:3] == 0).all() and nxt[3] >= 0


def test_a_millionth_is_greedy():
    """The fp32 number 1e-6 is below 1e-6: as temperature 0, drawn drafts and all."""
    rng = np.random.default_rng(44)
    n = 30
    x = torch.tensor(_peaked(rng, 3 * n, 200), dtype=torch.float32, device="cuda")
    y = torch.tensor(_peaked(rng, 3 * n, 200), dtype=torch.float32, device="cuda")
    tokens = torch.stack([x[::3].argmax(1) * 0, y[::3].argmax(1), x[::3].argmax(1)], 1).flatten().to(torch.int32)
    u = torch.rand(3 * n, device="cuda")
    for drafts in (None, y):
        a, b, c = (pkg.verify_sample(x, tokens, _i32([-1, 0, 0] * n), _i32(range(0, 3 * n + 1, 3)), u, 3, draft_logits=drafts,
                                     temperature=torch.full((n,), t, device="cuda")) for t in (0.0, 1e-6, 1e-7))
        assert all(torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]) for k in a)
        assert (a["n_accepted"] == 1).all() and (a["path"][:, 1] == 2).sum() > n // 2
