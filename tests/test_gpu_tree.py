"""Attention of draft trees and the commit of their accepted rows, against the
fp64 oracle.

Tolerances, derived before the first run: those of the causal operator (see
test_gpu_attn.py; n is the number of keys that a row sees).  The moved rows,
the lengths and everything read back: equal.
"""
import numpy as np
import pytest
import torch

import block_quantized_moe_layer_gb300 as pkg
from oracle import tree as ot
from tests.test_gpu_attn import HEADS, _cache, _np

pytestmark = pytest.mark.gpu


def _tree(rng, m, kind="random"):
    if kind == "chain":
        return list(range(-1, m - 1))
    if kind == "roots":  # every node follows the prefix
        return [-1] * m
    if kind == "star":
        return [-1] + [0] * (m - 1)
    return [-1][:m] + [int(rng.integers(-1 if kind == "forest" else 0, i)) for i in range(1, m)]


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _check(rng, hq, hk, D, lens, news, P, act=None, window=0, kind="random", q_scale=1.5, pad_q=0, stream=None, trees=None,
           wild=1.0, bad=False):
    act = pkg.ACT_BF16 if act is None else act
    bf = act == pkg.ACT_BF16
    pages, table, keys, values, n_pages = _cache(rng, lens, hk, D, P, wild=wild)
    trees = [_tree(rng, m, kind) for m in news] if trees is None else trees
    starts = np.concatenate([[0], np.cumsum(news)])
    T, max_len = int(starts[-1]), max(max(lens), 1)
    at = pkg.Attention(hq, hk, D, P, n_pages, T, len(lens), max_len, act=act, rot_dim=0, window=window)
    dt = torch.bfloat16 if bf else torch.float32
    q = torch.tensor(rng.normal(size=(T, hq, D + pad_q)) * q_scale, device="cuda").to(dt)[..., :D]
    lse = torch.full((T + 1, hq), 7.0, device="cuda")
    out = torch.full((T + 1, hq, D), 7.0, dtype=dt, device="cuda")
    parents = _i32([p for t in trees for p in t])
    args = (q, pages, _i32(starts), _i32(lens), table, max(max(news), 1), max_len)
    at.forward(*args, out=out[:T], lse=lse[:T], parents=parents, stream=stream)
    torch.cuda.synchronize()
    if bad:
        with pytest.raises(pkg.MoEError, match="parent"):
            at.status()
    else:
        at.status()
    again = at.forward(*args, parents=parents)
    torch.cuda.synchronize()
    assert torch.equal(out[:T], again)
    assert (out[T] == 7).all() and (lse[T] == 7).all()  # behind the last sequence
    got, got_lse, qn = _np(out), _np(lse), _np(q)
    sc = D ** -0.5
    for b, (n, m) in enumerate(zip(lens, news)):
        if m == 0:
            continue
        sl = slice(starts[b], starts[b + 1])
        want, wl, mag = ot.attention(qn[sl], keys[b], values[b], trees[b], window, sc)
        s_abs = sc * np.abs(qn[sl]).max() * np.abs(keys[b]).sum(-1).max() if n else 0.0
        e = (D + 4) * 2.0 ** -24 * s_abs
        n_vis = min(n, window) if window else n
        rel = np.expm1(2 * e) + 2.0 ** -20 + n_vis * 2.0 ** -24
        tol = mag * (rel + (2.0 ** -11 if bf else 0)) + np.abs(want) * (2.0 ** -8 if bf else 2.0 ** -23)
        if bf and n:
            tol += n_vis * 2.0 ** -17 * 2.0 ** -8 * np.abs(values[b]).max()
        err = np.abs(got[sl] - want)
        assert np.isfinite(got[sl]).all()
        assert (err <= tol).all(), (b, float((err - tol).max()), float((err / tol.clip(1e-30)).max()))
        seen = np.isfinite(wl)
        assert np.array_equal(np.isneginf(got_lse[sl]), ~seen)
        assert (got[sl][~seen] == 0).all()
        assert (np.abs(got_lse[sl][seen] - wl[seen]) <= rel + (2.0 ** -11 if bf else 0) + 2.0 ** -22 * (1 + np.abs(wl[seen]))).all()
    at.close()
    return got


@pytest.mark.parametrize("act", [pkg.ACT_F32, pkg.ACT_BF16])
@pytest.mark.parametrize("hq,hk,D,rot", HEADS)
def test_tree_small_and_ragged(hq, hk, D, rot, act):
    rng = np.random.default_rng(D + hq)
    _check(rng, hq, hk, D, [4, 300, 129], [4, 3, 1], 16, act)
    _check(rng, hq, hk, D, [1], [1], 64, act)
    _check(rng, hq, hk, D, [130, 64, 15], [2, 0, 5], 32, act, kind="forest")


@pytest.mark.parametrize("hq,hk,D,rot", HEADS)
@pytest.mark.parametrize("nodes", [13, 33, 64])
def test_tree_wide(hq, hk, D, rot, nodes):
    """All kernels: up to 16 rows, up to 256, more; trees across the end of a tile and of a page."""
    rng = np.random.default_rng(D + hq + nodes)
    _check(rng, hq, hk, D, [nodes, 128 + nodes // 2, 300], [nodes, nodes, nodes - 5], 16)
    _check(rng, hq, hk, D, [255 + nodes], [nodes], 128, kind="forest")


@pytest.mark.parametrize("kind", ["chain", "roots", "star"])
def test_tree_shapes(kind):
    rng = np.random.default_rng(3)
    for hq, hk, D in ((4, 2, 64), (16, 2, 128), (16, 1, 192), (3, 3, 256)):
        for m in (2, 7, 31, 32, 64):
            _check(rng, hq, hk, D, [m + 60, m], [m, m], 32, kind=kind)


@pytest.mark.parametrize("window", [1, 2, 5, 40, 200])
@pytest.mark.parametrize("hq,hk,D,rot", HEADS)
def test_tree_window(hq, hk, D, rot, window):
    rng = np.random.default_rng(window + D)
    _check(rng, hq, hk, D, [400, 9, 130], [4, 3, 1], 16, window=window)
    _check(rng, hq, hk, D, [400, 40, 63], [33, 40, 64][:2] + [60], 32, window=window)
    _check(rng, hq, hk, D, [300], [64], 64, window=window, kind="chain")
    if window < 50:
        _check(rng, hq, hk, D, [150], [9], 16, pkg.ACT_F32, window=window)


def test_tree_not_all_in_the_cache():
    """Fewer cached tokens than nodes: the first nodes see nothing and nobody sees them."""
    rng = np.random.default_rng(5)
    for hq, hk, D in ((2, 1, 64), (16, 2, 128), (16, 1, 192)):
        for act in (pkg.ACT_BF16, pkg.ACT_F32):
            _check(rng, hq, hk, D, [3, 0, 20], [8, 2, 33], 16, act)
            _check(rng, hq, hk, D, [3, 30], [8, 33], 16, act, kind="chain", window=4)


def test_tree_long_and_split():
    rng = np.random.default_rng(6)
    _check(rng, 4, 4, 128, [9001], [6], 16)
    _check(rng, 16, 1, 192, [5003], [16], 64)
    _check(rng, 16, 1, 192, [3000, 1500], [64, 30], 64)


def test_tree_chain_is_causal():
    """A chain gives the causal call's bits up to 64 rows, where the same kernel runs."""
    rng = np.random.default_rng(7)
    for hq, hk, D, m, window in ((16, 2, 128, 2, 0), (16, 2, 128, 8, 0), (16, 1, 192, 4, 0), (4, 1, 64, 4, 7), (2, 2, 256, 60, 90)):
        pages, table, _, _, n_pages = _cache(rng, [500, m], hk, D, 16)
        at = pkg.Attention(hq, hk, D, 16, n_pages, 2 * m, 2, 500, rot_dim=0, window=window)
        q = torch.tensor(rng.normal(size=(2 * m, hq, D)), device="cuda").to(torch.bfloat16)
        args = (q, pages, _i32([0, m, 2 * m]), _i32([500, m]), table, m, 500)
        one = at.forward(*args)
        two = at.forward(*args, parents=_i32(2 * list(range(-1, m - 1))))
        assert torch.equal(one, two)
        at.close()


def test_tree_strides_stream_and_values():
    rng = np.random.default_rng(8)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        _check(rng, 16, 2, 64, [300, 50], [4, 12], 16, pad_q=8)
    _check(rng, 16, 2, 128, [600], [12], 64, q_scale=30.0)
    _check(rng, 16, 2, 128, [600], [12], 64, q_scale=0.0)
    _check(rng, 16, 2, 192, [600], [40], 64, wild=60.0, q_scale=0.02)


def test_tree_bad_parents_are_reported():
    rng = np.random.default_rng(9)
    for hq, m in ((2, 5), (16, 12), (16, 40)):
        t = _tree(rng, m)
        t[1], t[2], t[3], t[4] = 1, m + 70, -2, 2 ** 31 - 1
        _check(rng, hq, 1, 64, [m + 20], [m], 16, trees=[t], bad=True)
        _check(rng, hq, 1, 64, [m + 20], [m], 16, pkg.ACT_F32, trees=[t], bad=True)


def test_tree_nan_query():
    rng = np.random.default_rng(10)
    for m in (3, 12, 40):
        pages, table, _, _, n_pages = _cache(rng, [100], 1, 128, 16)
        at = pkg.Attention(16, 1, 128, 16, n_pages, m, 1, 100, rot_dim=0)
        q = torch.tensor(rng.normal(size=(m, 16, 128)), device="cuda").to(torch.bfloat16)
        args = (pages, _i32([0, m]), _i32([100]), table, m, 100)
        good = at.forward(q, *args, parents=_i32(_tree(rng, m, "star")))
        q2 = q.clone()
        q2[1, 3] = float("nan")
        got = at.forward(q2, *args, parents=_i32(_tree(rng, m, "star")))
        assert got[1, 3].isnan().all()
        got[1, 3] = good[1, 3]
        assert torch.equal(got, good)
        at.close()


def test_tree_captured():
    rng = np.random.default_rng(11)
    m = 12
    pages, table, _, _, n_pages = _cache(rng, [700], 2, 128, 16)
    at = pkg.Attention(16, 2, 128, 16, n_pages, m, 1, 700, rot_dim=0)
    q = torch.tensor(rng.normal(size=(m, 16, 128)), device="cuda").to(torch.bfloat16)
    parents, lens, path = _i32(_tree(rng, m)), _i32([700]), _i32([[0, 3, 7, -1]])
    args = (pages, _i32([0, m]), lens, table)
    new = torch.empty_like(lens)
    at.forward(q, *args, m, 700, parents=parents)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = at.forward(q, *args, m, 700, parents=parents)
        at.commit(*args, path, 700, new_lens=new)
    other = [-1] + [0] * (m - 1)
    parents.copy_(_i32(other))
    before = pages.clone()
    g.replay()
    torch.cuda.synchronize()
    assert new.tolist() == [691]
    assert torch.equal(out, at.forward(q, before, *args[1:], m, 700, parents=_i32(other)))
    at.close()


@pytest.mark.parametrize("hq,m", [(2, 4), (16, 3), (16, 40)])
def test_tree_waits_run_out(hq, m):
    """Each kernel's bounded waits: reported, and later calls are unaffected."""
    rng = np.random.default_rng(12)
    pages, table, _, _, n_pages = _cache(rng, [500], 1, 128, 16)
    at = pkg.Attention(hq, 1, 128, 16, n_pages, m, 1, 500, rot_dim=0)
    q = torch.tensor(rng.normal(size=(m, hq, 128)), device="cuda").to(torch.bfloat16)
    args = (q, pages, _i32([0, m]), _i32([500]), table, m, 500)
    parents = _i32(_tree(rng, m))
    want = at.forward(*args, parents=parents)
    at.inject_timeout(1000)
    at.forward(*args, parents=parents)
    with pytest.raises(pkg.MoEError) as e:
        at.status()
    assert e.value.code == pkg.MOE_ETIMEOUT
    assert torch.equal(at.forward(*args, parents=parents), want)
    at.status()
    at.close()


def test_tree_around_the_row_limits():
    """The most rows of the verify kernel and one node more, with several row tiles of pairs."""
    rng = np.random.default_rng(13)
    for hq, hk, D, nodes in ((4, 1, 64, 32), (8, 2, 128, 32), (16, 1, 192, 8), (8, 1, 256, 8), (16, 2, 64, 16), (16, 1, 192, 33)):
        for m in (nodes, nodes + 1):
            _check(rng, hq, hk, D, [m + 300, m, 129 + m], [m, m, 1], 16)


@pytest.mark.parametrize("seqs,m,window", [(40, 9, 0), (12, 64, 0), (130, 5, 0), (130, 33, 0), (40, 9, 50)])
def test_tree_more_blocks_than_the_gpu_holds(seqs, m, window):
    """Calls that take the longest sequences first: lengths up and down, equal ones, sequences without nodes or tokens."""
    rng = np.random.default_rng(seqs + m)
    news = [int(x) for x in rng.integers(1, m + 1, seqs)]
    news[0], news[3], news[5] = m, 0, 0
    lens = [n + int(rng.choice([0, 7, 7, 64, 200, 330])) for n in news]
    lens[5] = 0
    _check(rng, 32, 8, 64, lens, news, 32, window=window)


@pytest.mark.parametrize("hq,hk,D,m", [(32, 8, 64, 4), (8, 2, 128, 4), (16, 1, 192, 1), (16, 2, 256, 2),
                                       (32, 8, 64, 12), (8, 2, 128, 32), (16, 1, 192, 8), (16, 2, 256, 8)])
def test_tree_parts_of_short_contexts(hq, hk, D, m):
    """Two to nine parts of a context, around the number that a cluster joins; sequences whose parts are mostly empty, or all."""
    rng = np.random.default_rng(D + m)
    for n in (129, 300, 513, 1024, 1030, 2049):
        _check(rng, hq, hk, D, [n], [m], 64)
        _check(rng, hq, hk, D, [n, m, m + 1, 0], [m, m, 1, 0], 64)
        _check(rng, hq, hk, D, [n, n - 50], [m, max(m - 1, 1)], 32, window=200)
    _check(rng, hq, hk, D, [600, 2], [m, m], 16)  # fewer cached tokens than nodes


# ------------------------------------------------------------------ commit


def _commit_check(rng, hk, D, P, lens, news, paths, width, ok=True, kept=None, pages=None):
    pages, table, _, _, n_pages = _cache(rng, lens, hk, D, P)
    at = pkg.Attention(hk, hk, D, P, n_pages, max(sum(news), 1), len(lens), max(max(lens), 1), act=pkg.ACT_F32, rot_dim=0)
    path = np.full((len(lens), width), -1)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    before = pages.clone()
    starts = np.concatenate([[0], np.cumsum(news)])
    new = at.commit(pages, _i32(starts), _i32(lens), table, _i32(path), max(max(lens), 1))
    torch.cuda.synchronize()
    if ok:
        at.status()
    else:
        with pytest.raises(pkg.MoEError):
            at.status()
    kept = paths if kept is None else kept
    want = before.cpu().numpy().reshape(n_pages, hk, -1)
    tb = table.cpu().numpy()
    from oracle import attn as oa
    src, dst = oa.page_arrays(before.cpu().numpy(), hk, P, D), oa.page_arrays(want, hk, P, D)
    lengths = []
    for b, (n, m, p) in enumerate(zip(lens, news, kept)):
        if p is None:
            lengths.append(n)
            continue
        j = np.arange(n)
        for s, d in zip(src, dst):
            rows, length = ot.committed(s[tb[b, j // P], :, j % P], m, p)
            d[tb[b, j // P], :, j % P] = rows
        lengths.append(length)
    assert new.tolist() == lengths
    assert np.array_equal(pages.cpu().numpy(), want.reshape(n_pages, -1))
    at.close()


@pytest.mark.parametrize("hk,D", [(1, 64), (8, 128), (4, 192), (2, 256)])
@pytest.mark.parametrize("P", [16, 64])
def test_commit(hk, D, P):
    rng = np.random.default_rng(D + P)
    lens = [100, 64, 17, 1, 0, 333, 200]
    news = [64, 64, 5, 1, 0, 40, 0]
    paths = [sorted(rng.choice(64, 20, replace=False)), list(range(64)), [0, 2, 3, 4], [0], [], list(range(3, 40)), []]
    _commit_check(rng, hk, D, P, lens, news, paths, 64)
    # overlapping moves: each target is the source of an earlier place
    _commit_check(rng, hk, D, P, [90, 40], [30, 12], [list(range(1, 30)), list(range(0, 12, 2))], 29)
    _commit_check(rng, hk, D, P, [90], [30], [[]], 1)
    _commit_check(rng, hk, D, P, [90], [30], [[29]], 1)


def test_commit_reports():
    rng = np.random.default_rng(1)
    lens, news = [50, 60, 70, 20], [10, 10, 10, 5]
    _commit_check(rng, 2, 64, 16, lens, news, [[0, 3, 10], [4, 4], [5, 2, 7], [-2]], 3, False, [[0, 3], [4], [5], []])
    # more nodes than tokens, more nodes than a tree has
    _commit_check(rng, 2, 64, 16, [5, 90], [8, 65], [[0, 2], [0, 2]], 2, False, [None, None])


def test_commit_length_and_pages_out_of_range():
    rng = np.random.default_rng(2)
    pages, table, _, _, n_pages = _cache(rng, [40], 2, 64, 16)
    at = pkg.Attention(2, 2, 64, 16, n_pages, 10, 1, 40, act=pkg.ACT_F32, rot_dim=0)
    before = pages.clone()
    for n in (41, -1):
        assert at.commit(pages, _i32([0, 10]), _i32([n]), table, _i32([[0, 5]]), 40).tolist() == [n]
        with pytest.raises(pkg.MoEError, match="lengths"):
            at.status()
    for entry in (-1, n_pages, 2 ** 31 - 1):
        bad = table.clone()
        bad[0, 2] = entry  # rows 32..39: the nodes 2..9
        assert at.commit(pages, _i32([0, 10]), _i32([40]), bad, _i32([[0, 5]]), 40).tolist() == [32]
        with pytest.raises(pkg.MoEError, match="block-table"):
            at.status()
    assert torch.equal(pages, before)
    at.close()


def test_refusals():
    at = pkg.Attention(2, 1, 64, 16, 8, 100, 4, 128, rot_dim=0)
    q = torch.zeros(70, 2, 64, dtype=torch.bfloat16, device="cuda")
    pages, table, lens = at.pages(), _i32(np.arange(8)[None]), _i32([100])
    with pytest.raises(pkg.MoEError, match="at most 64"):
        at.forward(q, pages, _i32([0, 70]), lens, table, 70, 100, parents=_i32([-1] * 70))
    for parents in (_i32([-1] * 69), torch.full((70,), -1, device="cuda"), torch.full((70,), -1, dtype=torch.int32), _i32([-1] * 140)[::2]):
        with pytest.raises(pkg.MoEError, match="parents"):
            at.forward(q, pages, _i32([0, 70]), lens, table, 64, 100, parents=parents)
    starts, path = _i32([0, 4]), _i32([[0, 2]])
    for args, what in (((pages, starts, lens, table, _i32([0, 2]), 100), "path"), ((pages, starts, lens, table, path.long(), 100), "path"),
                       ((pages, starts[:1], lens, table, path, 100), "starts"), ((pages, starts, lens.long(), table, path, 100), "lens"),
                       ((pages, starts, lens, table, path, 129), "max_len"), ((pages[:3], starts, lens, table, path, 100), "pages"),
                       ((pages, starts, lens, table, _i32([[-1] * 65]), 100), "path_width")):
        with pytest.raises(pkg.MoEError, match=what):
            at.commit(*args)
    with pytest.raises(pkg.MoEError, match="overlap"):
        at.commit(pages, starts, lens, table, path, 100, new_lens=lens)
    at.close()
