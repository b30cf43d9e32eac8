"""Sampled verification of siblings drawn without replacement where a few tokens
hold nearly all of the draft head's probability: what is left of it is a small
part of a row's sum, and the later siblings are judged by shares of that part.

The outcomes are chosen with room: a number differs from the border of its
outcome by 2^-10 of it at least (asserted), so every path and token is equal to
the fp64 oracle's.
"""
import numpy as np
import pytest
import torch

import block_quantized_moe_layer_gb300 as pkg
from oracle import tree as ot
from tests.test_gpu_verify_sample import _i32

pytestmark = pytest.mark.gpu


def _check(x, y, tokens, trees, uniforms, dtype, temperature=None):
    """Rows x, y of all nodes; trees and their numbers of nodes; every sequence is compared."""
    sizes = [len(t) for t in trees]
    starts = np.concatenate([[0], np.cumsum(sizes)])
    xd, yd = (torch.tensor(a, dtype=torch.float32, device="cuda").to(dtype) for a in (x, y))
    u = np.asarray(uniforms, np.float32)
    t = np.ones(len(sizes), np.float32) if temperature is None else np.asarray(temperature, np.float32)
    r = pkg.verify_sample(xd, _i32(tokens), _i32([p for s in trees for p in s]), _i32(starts), torch.tensor(u, device="cuda"), max(sizes),
                          draft_logits=yd, temperature=torch.tensor(t, device="cuda"))
    path, acc, nxt = (r[k].cpu().numpy() for k in ("path", "n_accepted", "next"))
    xs, ys = xd.double().cpu().numpy(), yd.double().cpu().numpy()
    taken = []
    for b in range(len(sizes)):
        s = slice(starts[b], starts[b + 1])
        want, token, gap = ot.verify(xs[s], np.asarray(tokens)[s], trees[b], u[s].astype(np.float64), ys[s], float(t[b]))
        assert gap > 2.0 ** -10, (b, gap)
        got = path[b][path[b] >= 0].tolist()
        assert (got, acc[b], nxt[b]) == (want, len(want) - 1, token), (b, got, want, nxt[b], token)
        taken.append(want)
    return taken


def _rows(rng, V, bits, p2, q2, third):
    """Rows (x, y) of one sequence of a root and three children, and their tokens: q(x1) = 1 - 2^-bits, of the rest
    q2 is x2's; p is mostly the third token's (`third` of it) and p2 x2's."""
    a, b, c = (int(v) for v in rng.choice(V, 3, replace=False))
    y = rng.normal(size=(4, V))
    x = rng.normal(size=(4, V))
    others = np.ones(V, bool)
    others[[a, b, c]] = False
    total = np.exp(y[0, others]).sum()
    y[0, c] = np.log(total * 0.5)
    total *= 1.5
    y[0, b] = np.log(total * q2 / (1 - q2))
    total /= 1 - q2
    y[0, a] = np.log(total) + bits * np.log(2.0)
    rest = 1 - third - p2 - 0.001
    x[0, others] += np.log(rest) - np.log(np.exp(x[0, others]).sum())
    x[0, a], x[0, b], x[0, c] = np.log(0.001), np.log(p2), np.log(third)
    x[1:, c] = np.log(V) + 8  # (the rows after the children: one token)
    return x, y, [0, a, b, c]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n_seqs", [(50, 108), (4099, 60), (20011, 2), (151936, 18)])
def test_siblings_of_a_peaked_draft(V, n_seqs, dtype):
    rng = np.random.default_rng(V)
    xs, ys, tokens, numbers = [], [], [], []
    b = 0
    while len(xs) < n_seqs:
        bits = 20 + b * 7 % 41
        p2 = (0.5, 0.01, 1e-6)[b % 3]
        q2 = (0.6, 0.05)[b // 3 % 2]
        x, y, t = _rows(rng, V, bits, p2, q2, 0.45 if p2 == 0.5 else 0.9)
        # the second sibling's number on either side of p2 / q2, which is its border (up to the rest)
        border = min(p2 / q2, 1.0)
        u = [rng.uniform(0.1, 0.9), 0.5, border * (0.5, 1.5)[b // 2 % 2] if border < 0.6 else (0.3, 0.95)[b // 2 % 2], rng.uniform(0.05, 0.5)]
        b += 1
        xr, yr = (torch.tensor(a, dtype=torch.float32).to(dtype).double().numpy() for a in (x, y))
        if ot.verify(xr, t, [-1, 0, 0, 0], np.asarray(u, np.float32).astype(np.float64), yr)[2] <= 2.0 ** -9:
            continue  # (another input, before the operator has seen it)
        xs.append(x), ys.append(y), tokens.extend(t), numbers.extend(u)
    taken = _check(np.concatenate(xs), np.concatenate(ys), tokens, [[-1, 0, 0, 0]] * n_seqs, numbers, dtype)
    assert all(t[1:] != [1] for t in taken)
    if n_seqs > 10:
        assert {tuple(t) for t in taken} == {(0, 2), (0, 3)}


def test_a_row_of_powers():
    """Siblings each of which holds nearly all that the ones before it left: twelve of them, down to 2^-396 of the row."""
    rng = np.random.default_rng(1)
    V, n = 3000, 12
    for step in (4, 20, 33):  # bits from one sibling to the next
        for offset in (0.0, 5000.0, -5000.0):
            xs, ys, tokens, numbers = [], [], [], []
            for b in range(16):
                ids = rng.choice(V, n, replace=False)
                y = np.full((n + 1, V), -step * (n + 1) * np.log(2.0)) - np.log(V)
                y[:, ids] = -step * np.arange(n) * np.log(2.0)
                x = rng.normal(size=(n + 1, V)) - 8
                x[:, ids[b % n]] = 5.0  # what the target wants: one of them
                u = rng.uniform(0.3, 0.7, n + 1)
                xs.append(x), ys.append(y + offset), tokens.extend([0] + ids.tolist()), numbers.extend(u)
            taken = _check(np.concatenate(xs), np.concatenate(ys), tokens, [[-1] + [0] * n] * 16, numbers, torch.float32)
            assert [t[1:] for t in taken] == [[b % n + 1] for b in range(16)]


def test_nothing_left_of_the_draft():
    """Less than 2^-400 of the draft row's largest is left: the later siblings are passed over; with more they are judged."""
    V = 60
    x = np.zeros((3, V))
    x[0, 7], x[0, 9] = 2.0, -3.0
    for gap, judged in ((200.0, True), (275.0, True), (280.0, False), (2000.0, False), (np.inf, False)):
        for offset in (0.0, 20000.0):
            y = np.full((3, V), -gap) + offset
            y[:, 9] = offset
            # the first sibling is rejected; the second one's share of what is left is 1/59, less than the target's
            taken = _check(x, y, [0, 9, 7], [[-1, 0, 0]], [0.508, 0.9, 0.9], torch.float32)
            assert taken == [[0, 2] if judged else [0]], (gap, offset)


@pytest.mark.parametrize("bits", [20, 34, 40, 60])
def test_tokens_are_distributed_as_the_target(bits):
    """The token after the root over many sequences whose draft row is nearly one token: each frequency within 5 standard deviations of p."""
    n, V = 40000, 6
    g = torch.Generator(device="cuda").manual_seed(bits)
    p = torch.tensor([-2.0, -1.0, 1.5, 0.0, -6.0, 0.3], device="cuda")
    q = torch.tensor([0.0, 2.5, -1.0, 0.5, 1.0, -0.5], device="cuda")
    q[0] = bits * np.log(2.0)
    pq = torch.softmax(q.double(), 0)
    # draws without replacement: the smallest of exponential numbers over the probabilities
    kids = (torch.empty(n, V, dtype=torch.float64, device="cuda").exponential_(generator=g) / pq).topk(3, 1, largest=False).indices
    tokens = torch.cat([torch.zeros(n, 1, device="cuda"), kids], 1).to(torch.int32).reshape(-1)
    r = pkg.verify_sample(p.expand(4 * n, V).contiguous(), tokens, _i32([-1, 0, 0, 0]).repeat(n),
                          torch.arange(0, 4 * n + 1, 4, dtype=torch.int32, device="cuda"), torch.rand(4 * n, generator=g, device="cuda"), 4,
                          draft_logits=q.expand(4 * n, V).contiguous())
    took = r["path"][:, 1].long()
    first = torch.where(took > 0, tokens.view(n, 4).gather(1, took.clamp(min=0)[:, None])[:, 0].long(), r["next"].long())
    share = torch.bincount(first, minlength=V).double() / n
    want = torch.softmax(p.double(), 0)
    assert ((share - want).abs() <= 5 * (want * (1 - want) / n).sqrt()).all(), (share, want)
    assert (took > 1).float().mean() > 0.2  # (later siblings are accepted)
