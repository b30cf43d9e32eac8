"""fp64 oracle of the attention operators: the 4-bit page format, the append
step (norms, rotation, codes), paged causal attention, and token scores.

Plain numpy from the definitions in ``moe_layer.h``; nothing here calls or
imports the GPU path.
"""
import numpy as np

KV_MAX_SCALE = 198


def scale_of(b):
    """The scale a byte stands for: 5 exponent bits, 3 fraction bits, bias 15."""
    b = np.asarray(b, np.int64)
    e, m = b >> 3, (b & 7).astype(np.float64)
    return np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 15), m / 8 * 2.0 ** -14)


_GRID = scale_of(np.arange(KV_MAX_SCALE + 1))


def quantise(x):
    """Codes 0..15 [..., D] and scale bytes [..., D/16] of rows x [..., D]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    g = np.where(np.isnan(g), 0.0, g)
    v = np.abs(g).max(-1) / 7
    hi = np.clip(np.searchsorted(_GRID, v), 1, KV_MAX_SCALE)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        b = np.where(v - _GRID[lo] < _GRID[hi] - v, lo, hi)
        tie = v - _GRID[lo] == _GRID[hi] - v
    b = np.where(tie, np.where(lo % 2 == 0, lo, hi), b)
    b = np.where(v >= _GRID[-1], KV_MAX_SCALE, b)
    d = scale_of(b)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(d > 0, np.clip(np.rint(g / d), -8, 7), 0.0) + 8
    return c.astype(np.uint8).reshape(x.shape), b.astype(np.uint8)


def dequantise(codes, scales):
    c = codes.astype(np.float64).reshape(codes.shape[:-1] + (codes.shape[-1] // 16, 16)) - 8
    return (c * scale_of(scales)[..., None]).reshape(codes.shape)


def pack(codes):
    """Codes [..., D] -> bytes [..., D/2]: channel e of eight is nibble e/2 + 4 (e%2)."""
    c = codes.reshape(codes.shape[:-1] + (-1, 8)).astype(np.uint32)
    w = np.zeros(c.shape[:-1], np.uint32)
    for e in range(8):
        w |= c[..., e] << np.uint32(4 * (e // 2 + 4 * (e % 2)))
    return np.ascontiguousarray(w).astype("<u4").view(np.uint8).reshape(codes.shape[:-1] + (-1,))


def unpack(b):
    w = np.ascontiguousarray(b).view("<u4")
    c = np.stack([(w >> np.uint32(4 * (e // 2 + 4 * (e % 2)))) & 15 for e in range(8)], -1)
    return c.reshape(b.shape[:-1] + (-1,)).astype(np.uint8)


def page_arrays(pages, hk, P, D):
    """Views (key codes, key scales, value codes, value scales) [page, head, token, bytes] of a page buffer."""
    n = pages.shape[0]
    rows = pages.reshape(n, hk, P * D * 9 // 8)
    out, at = [], 0
    for w in (D // 2, D // 16, D // 2, D // 16):
        out.append(rows[:, :, at:at + P * w].reshape(n, hk, P, w))
        at += P * w
    return out


def prepared(x, w, pos, rot, freq, interleaved=False, eps=1e-6):
    """Normalised (w not None) and rotated rows x [T, heads, D] at positions pos."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    if rot:
        a = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
        c, s = np.cos(a), np.sin(a)
        x = x.copy()
        i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        p, q = x[..., i].copy(), x[..., j].copy()
        x[..., i], x[..., j] = p * c - q * s, q * c + p * s
    return x


def frequencies(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot) if rot else np.zeros(0)


def attention(q, keys, values, n_new, window=0, scale=None):
    """One sequence: q [n_new, hq, D] the last n_new of len(keys) tokens, keys
    and values [len, hk, D].  Returns (out [n_new, hq, D], lse [n_new, hq],
    mag [n_new, hq, D]: the softmax-weighted |v|, for error bounds)."""
    q = np.asarray(q, np.float64)
    n, hk, D = keys.shape
    hq = q.shape[1]
    g = hq // hk
    scale = D ** -0.5 if scale is None else scale
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    for t in range(n_new):
        pos = n - n_new + t
        lo = max(0, pos - window + 1) if window else 0
        if pos < lo:
            continue
        for h in range(hq):
            s = keys[lo:pos + 1, h // g] @ q[t, h] * scale
            m = s.max()
            p = np.exp(s - m)
            v = values[lo:pos + 1, h // g]
            out[t, h] = p @ v / p.sum()
            mag[t, h] = p @ np.abs(v) / p.sum()
            lse[t, h] = m + np.log(p.sum())
    return out, lse, mag


def scores(logits, tokens, n_top):
    """(logprob, entropy, top ids, top logprobs) of rows of logits; a row without a logit above -inf as documented."""
    x = np.asarray(logits, np.float64)
    n = x.shape[0]
    lp, en = np.full(n, np.nan), np.zeros(n)
    ids = np.argsort(-x, axis=1, kind="stable")[:, :n_top]
    tl = np.full(ids.shape, -np.inf)
    for i in range(n):
        m = x[i].max()
        ok = 0 <= tokens[i] < x.shape[1]
        if m == -np.inf:
            if ok:
                lp[i] = -np.inf
            continue
        z = x[i] - m
        e = np.exp(z)
        ls = np.log(e.sum())
        en[i] = ls - (e * np.where(e > 0, z, 0.0)).sum() / e.sum()
        if ok:
            lp[i] = z[tokens[i]] - ls
        tl[i] = z[ids[i]] - ls
    return lp, en, ids, tl
