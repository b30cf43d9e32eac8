"""Pins of the tree operators' oracle: hand-worked examples and the causal one."""
import numpy as np

from oracle import attn as oa
from oracle import tree as ot


def test_lines_and_visible_rows():
    parents = [-1, 0, 0, 2, 7, -1]
    assert ot.line(parents, 3) == [3, 2, 0] and ot.line(parents, 4) == [4] and ot.line(parents, 5) == [5]
    rows = ot.visible(parents, 8)
    assert rows[3] == [5, 4, 2, 1, 0] and rows[5] == [7, 1, 0]
    assert ot.visible(parents, 8, 2)[3] == [5, 4] and ot.visible(parents, 8, 4)[3] == [5, 4, 2, 1]
    assert ot.visible(parents, 4)[:4] == [[], [], [0], [1, 0]]


def test_chain_is_causal():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(5, 4, 16)), rng.normal(size=(20, 2, 16)), rng.normal(size=(20, 2, 16))
    for window in (0, 3, 9):
        for a, b in zip(ot.attention(q, k, v, range(-1, 4), window), oa.attention(q, k, v, 5, window)):
            assert np.allclose(a, b, atol=1e-12)


def test_verify_by_hand():
    log = np.log
    p = log(np.array([[0.5, 0.25, 0.25], [0.1, 0.2, 0.7], [1.0, 1.0, 1.0]]))
    # the child's token has p = 0.25
    assert ot.verify(p, [0, 1, 0], [-1, 0, 1], [0.1, 0.24, 0.99])[:2] == ([0, 1], 1)  # then 0.99 > 0.1; 0.1 of 0.9 without token 0
    assert ot.verify(p, [0, 1, 0], [-1, 0, 1], [0.7, 0.26, 0.0])[:2] == ([0], 2)  # 0.7 of 0.75: past token 0's 0.5
    # drawn from q = (0.1, 0.8, 0.1): u q < p; the rest is (0.4, 0, 0.15)
    q = log(np.array([[0.1, 0.8, 0.1]] * 3))
    assert ot.verify(p, [0, 1, 0], [-1, 0, 1], [0.0, 0.31, 0.5], q)[0] == [0, 1, 2]
    assert ot.verify(p, [0, 1, 0], [-1, 0, 1], [0.72, 0.32, 0.5], q)[:2] == ([0], 0)
    assert ot.verify(p, [0, 1, 0], [-1, 0, 1], [0.74, 0.32, 0.5], q)[:2] == ([0], 2)
    assert ot.verify(p, [0, 0, 0], [-1, 0, 1], [0.5, 0.9, 0.9], temperature=0.0)[:2] == ([0, 1], 2)


def test_commit_by_hand():
    rows, n = ot.committed(np.arange(10), 6, [0, 2, 3])
    assert rows.tolist() == [0, 1, 2, 3, 4, 6, 7, 7, 8, 9] and n == 7
