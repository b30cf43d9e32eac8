"""fp64 oracle of the operators on trees of drafted tokens: attention of a
tree's nodes, sampled verification, the cache rows that stay.

Plain numpy from the definitions in ``moe_layer.h``; nothing here calls or
imports the GPU path.
"""
import numpy as np


def line(parents, i):
    """Node i and its ancestors, upwards.  A parent that is no earlier node counts as -1."""
    out = [i]
    while 0 <= parents[i] < i:
        i = parents[i]
        out.append(i)
    return out


def visible(parents, n, window=0):
    """For each node the cache rows it sees, of n cached tokens whose last len(parents) are the nodes."""
    first = n - len(parents)
    rows = []
    for i in range(len(parents)):
        if first + i < 0:
            rows.append([])
            continue
        seen = [first + a for a in line(parents, i)] + list(range(first - 1, -1, -1))
        rows.append([j for j in (seen[:window] if window else seen) if j >= 0])
    return rows


def attention(q, keys, values, parents, window=0, scale=None):
    """One sequence: q [m, hq, D] of the m nodes, keys and values [n, hk, D]:
    (out, lse, mag) as :func:`oracle.attn.attention` gives them."""
    q = np.asarray(q, np.float64)
    n, hk, D = keys.shape
    g = q.shape[1] // hk
    scale = D ** -0.5 if scale is None else scale
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    for i, rows in enumerate(visible(parents, n, window)):
        if not rows:
            continue
        for h in range(q.shape[1]):
            s = keys[rows, h // g] @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            v = values[rows, h // g]
            out[i, h] = p @ v / p.sum()
            mag[i, h] = p @ np.abs(v) / p.sum()
            lse[i, h] = m + np.log(p.sum())
    return out, lse, mag


def distribution(logits, temperature=1.0):
    """Probabilities of a row, or None where it has no distribution."""
    x = np.asarray(logits, np.float64)
    if not 0 <= temperature <= 1e6 or np.isnan(x).any() or x.max() in (np.inf, -np.inf):
        return None
    if temperature < 1e-6:
        p = np.zeros(len(x))
        p[int(np.flatnonzero(x == x.max())[0])] = 1
        return p
    e = np.exp((x - x.max()) / temperature)
    return e / e.sum()


def verify(logits, tokens, parents, uniforms, draft_logits=None, temperature=1.0, replacement=False):
    """One sequence: (accepted path, next token, least distance of a number to
    the border of its outcome, relative to the whole)."""
    V, m = np.asarray(logits).shape[1], len(tokens)
    path, gap = [0], np.inf
    greedy = temperature < 1e-6
    while True:
        at = path[-1]
        p = distribution(logits[at], temperature)
        if p is None:
            return path, -1, gap
        q = None
        children = [i for i in range(at + 1, m) if parents[i] == at]
        if draft_logits is not None and not greedy:
            q = distribution(draft_logits[at], temperature)
            if q is None:
                children = []
        r, had, taken = p.copy(), set(), None
        if q is not None:
            rest, whole = q.copy(), q.max()  # what is left of q, and its largest at first
        for i in children:
            x, u = int(tokens[i]), float(uniforms[i])
            if not 0 <= x < V or (x in had and not (q is not None and replacement)):
                continue
            had.add(x)
            total = r.sum()
            side = u * total * (1.0 if q is None else q[x])
            gap = min(gap, abs(side - r[x]) / max(side, r[x], 1e-300)) if max(side, r[x]) > 0 else gap
            if side < r[x]:
                taken = i
                break
            if q is None:
                r[x] = 0
            elif total > 0 and q.sum() > 0:
                r = np.maximum(r / total - q, 0)
                if not replacement:
                    rest[x] = 0
                    if not rest.max() > 2.0 ** -400 * whole:
                        break  # nothing is left of q: the later siblings are passed over
                    q = rest / rest.sum()
        if taken is not None:
            path.append(taken)
            continue
        if not r.sum() > 0:
            r = p
        mass = np.cumsum(r)
        t = float(uniforms[0]) * mass[-1]
        v = int(np.searchsorted(mass, t, side="right"))
        v = min(v, int(np.flatnonzero(r > 0)[-1]))
        gap = min(gap, abs(mass[v] - t) / mass[-1], abs(t - (mass[v - 1] if v else 0)) / mass[-1] if v else np.inf)
        return path, v, gap


def committed(rows, m, path):
    """The cache rows [n, ...] of a sequence with m nodes after its path is kept, and its new length."""
    first = len(rows) - m
    out = rows.copy()
    for k, i in enumerate(path):
        out[first + k] = rows[first + i]
    return out, first + len(path)
