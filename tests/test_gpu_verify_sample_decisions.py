"""Every decision of a walk against the definition, none left out: a draft is
accepted, or rejected, and the next token's place taken, within the documented
errors of the row's sums (2^-32, and 2^-31 more for each rejected draft; of a drawn
draft's share of what is left, 2^-30), where the other decisions are as they were
made.  Numbers of 0 and 1 - 2^-24 are frequent, drafts arbitrary.
"""
import numpy as np
import pytest
import torch

import block_quantized_moe_layer_gb300 as pkg
from oracle import tree as ot
from tests.test_gpu_verify_sample import _i32

pytestmark = pytest.mark.gpu

ONE = 1 - 2.0 ** -24


def _wrong(x, tokens, parents, u, y, T, replacement, path, acc, nxt):
    """What is wrong with one sequence's outcome, or None."""
    V, m = x.shape[1], len(tokens)
    if path[0] != 0 or acc != len(path) - 1:
        return "path"
    greedy = T < 1e-6
    for at, took in zip(path, path[1:] + [None]):
        p = ot.distribution(x[at], T)
        if p is None:
            return None if took is None and nxt == -1 else "no distribution"
        q = None if y is None or greedy else ot.distribution(y[at], T)
        kids = [i for i in range(at + 1, m) if parents[i] == at] if y is None or greedy or q is not None else []
        r, had, room = p.copy(), set(), 2.0 ** -32
        if q is not None:
            rest, least = q.copy(), 2.0 ** -400 * q.max()
        for i in kids:
            v = int(tokens[i])
            if not 0 <= v < V or (v in had and not (q is not None and replacement)):
                continue
            had.add(v)
            total = r.sum()
            side = u[i] * total * (1.0 if q is None else q[v])
            # (u total q' takes the errors of total and of the share, relative ones)
            over = side - r[v]
            if i == took:
                if over > room + 2.0 ** -29 * side:
                    return "accepted", i, side, r[v]
                break
            if -over > room + 2.0 ** -29 * side:
                return "rejected", i, side, r[v]
            if q is None:
                r[v] = 0
            else:
                r = np.maximum(r - total * q, 0)
                if not replacement:
                    rest[v] = 0
                    if not rest.max() > least:
                        break
                    q = rest / rest.sum()
            room += 2.0 ** -31
        else:
            if took is not None:
                return "went on", took
        if took is not None:
            if took not in kids:
                return "went on", took
            continue
        if not (0 <= nxt < V and p[nxt] > 0):
            return "next", nxt
        total, mass = r.sum(), np.cumsum(r)
        if total <= 4 * room:
            continue  # (about nothing is left: any token of p)
        t = u[0] * total
        if not mass[nxt] - r[nxt] - 2 * room <= t <= mass[nxt] + 2 * room or (q is None and not greedy and nxt in had):
            return "place", nxt, mass[nxt] - r[nxt], t, mass[nxt]
    return None


def _inputs(rng, mode, N, V):
    x = rng.normal(size=(N, V)) * 10.0 ** rng.uniform(-3, 1)
    y = x + rng.normal(size=(N, V)) * 10.0 ** rng.uniform(-6, 1)
    if mode == "huge":
        s = 10.0 ** rng.uniform(0, 37) / max(np.abs(x).max(), np.abs(y).max())
        x, y = x * s, y * s
    elif mode == "masked":
        x[rng.random((N, V)) < 0.8] = -np.inf
        y[rng.random((N, V)) < 0.8] = -np.inf
        x[:, -1] = y[:, -1] = 0
    elif mode == "ties":
        x, y = np.round(x * 2) / 2, np.round(y * 2) / 2
    elif mode == "peaked":
        x[np.arange(N), rng.integers(0, V, N)] += rng.uniform(0, 40, N)
        y = np.where(rng.random((N, 1)) < 0.5, x, y)
        y[np.arange(N), rng.integers(0, V, N)] += rng.uniform(0, 60, N)
    elif mode == "flat":
        x = np.full((N, V), float(rng.integers(-2, 3)))
        y = x.copy()
        y[:, rng.integers(0, V)] += rng.uniform(-5, 30)
    return x, y


@pytest.mark.parametrize("drafts", ["chosen", "drawn", "independent"])
@pytest.mark.parametrize("mode", ["any temperature", "huge", "masked", "ties", "peaked", "flat"])
def test_every_decision(mode, drafts):
    rng = np.random.default_rng([ord(c) for c in mode + drafts])
    drawn, replacement = drafts != "chosen", drafts == "independent"
    for call in range(40):
        V = int(rng.integers(*[(1, 20), (20, 300), (300, 9000), (9000, 40000)][call % 4]))
        sizes = [int(rng.integers(1, 9)) for _ in range(16 if V < 3000 else 3)]
        N, starts = sum(sizes), np.concatenate([[0], np.cumsum(sizes)])
        dtype = torch.bfloat16 if call % 3 == 0 else torch.float32
        low, high = (1.5e-6, 1e6) if mode == "any temperature" else (0.05, 3.0)
        T = np.exp(rng.uniform(np.log(low), np.log(high), len(sizes))).astype(np.float32)
        x, y = (torch.tensor(a, dtype=torch.float32, device="cuda").to(dtype) for a in _inputs(rng, mode, N, V))
        xs, ys = x.double().cpu().numpy(), y.double().cpu().numpy()
        trees = [[-1] + [int(rng.integers(max(0, (i - 1) // 4), min(i, (i - 1) // 3 + 1))) for i in range(1, m)] for m in sizes]
        tokens = rng.integers(-1, V + 1, N)
        if call % 2:  # likely ones
            best = np.argsort(-(ys if drawn else xs), 1)[:, :4]
            for b, t in enumerate(trees):
                for i, p in enumerate(t):
                    if p >= 0:
                        tokens[starts[b] + i] = best[starts[b] + p, rng.integers(best.shape[1])]
        u, kind = rng.random(N).astype(np.float32), rng.random(N)
        u[kind < 0.3] = 0
        u[kind > 0.75] = ONE
        u = np.minimum(u, np.float32(ONE))
        r = pkg.verify_sample(x, _i32(tokens), _i32([p for t in trees for p in t]), _i32(starts), torch.tensor(u, device="cuda"), max(sizes),
                              draft_logits=y if drawn else None, temperature=torch.tensor(T, device="cuda"), replacement=replacement)
        path, acc, nxt = (r[k].cpu().numpy() for k in ("path", "n_accepted", "next"))
        for b in range(len(sizes)):
            s = slice(starts[b], starts[b + 1])
            wrong = _wrong(xs[s], tokens[s], trees[b], u[s].astype(np.float64), ys[s] if drawn else None, float(T[b]), replacement,
                           path[b][path[b] >= 0].tolist(), int(acc[b]), int(nxt[b]))
            assert wrong is None, (call, b, V, float(T[b]), wrong)
