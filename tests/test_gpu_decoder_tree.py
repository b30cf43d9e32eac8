"""A tree of drafts through the decoder: append, attention, sampled verification,
commit and scores as a serving loop runs them."""
import numpy as np
import pytest
import torch

from block_quantized_moe_layer_gb300 import MoEError
from oracle import attn as oa
from oracle import tree as ot
from tests.test_gpu_decoder import _model, _np

pytestmark = pytest.mark.gpu

PARENTS = [0, 0, 1, 1, 2, 3]


def _rows(model, seq, n):
    j = torch.arange(n, device="cuda")
    slots = torch.tensor(seq.pages, device="cuda")[j // 16] * 16 + j % 16
    return model.block.attention.read(slots, model.block.cache)


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("temperature", [0.0, 0.7])
def test_tree_step(window, temperature):
    model = _model(window)
    at = model.block.attention
    seq = model.new_sequence()
    model.prefill(seq, np.random.default_rng(0).integers(0, 1000, 190).tolist())
    ahead = model._run(seq, [3])
    seq.length -= 1
    best = model._logits(ahead)[0].topk(2).indices.tolist()
    seen = {}
    forward, commit = at.forward, at.commit
    at.forward = lambda q, *a, **k: seen.setdefault("o", forward(seen.setdefault("q", q.clone()), *a, **k))
    at.commit = lambda pages, *a, **k: seen.setdefault("rows", _rows(model, seq, 197)) and commit(pages, *a, **k)
    numbers = np.linspace(0.05, 0.6, 7).astype(np.float32)
    r = model.verify_tree(seq, 3, best + [11, 12, 13, 14], PARENTS, uniforms=numbers.tolist(), temperature=temperature)
    del at.forward, at.commit
    keys, values = (_np(t) for t in seen["rows"])
    tree = [-1] + PARENTS
    want, _, mag = ot.attention(_np(seen["q"]), keys, values, tree, window)
    # a rounding of the output (2^-8), of the weights (2^-11) and of exponentials and sums (2^-17 here)
    assert (np.abs(_np(seen["o"]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mag).all()
    tokens = [3] + best + [11, 12, 13, 14]
    path, nxt, gap = ot.verify(_np(r["logits"]), tokens, tree, numbers.astype(np.float64), temperature=temperature)
    assert gap > 2.0 ** -26  # (of these fixed numbers)
    assert r["path"] == path and r["accept"] == [len(path) - 1, nxt] and seq.length == 190 + len(path)
    after = _rows(model, seq, 197)
    for a, b in zip((keys, values), after):
        assert np.array_equal(ot.committed(a, 7, path)[0], _np(b))
    checked = [tokens[i] for i in path[1:]] + [nxt]
    lp, _, ids, _ = oa.scores(_np(r["logits"])[path], checked, 4)
    assert np.allclose(_np(r["scores"]["logprob"]), lp, atol=1e-5) and np.array_equal(r["scores"]["top_ids"].cpu().numpy(), ids)
    if temperature == 0:
        assert path[1] == 1 and r["accept"][0] >= 1  # the best token is the first child
    at.status()


def test_a_chain_is_a_verify_step():
    """A tree that is a chain, at temperature 0, gives the bits of the greedy step of the same drafts."""
    a, b = _model(), _model()
    sa, sb = a.new_sequence(), b.new_sequence()
    for model, seq in ((a, sa), (b, sb)):
        model.prefill(seq, list(range(100, 200)))
    best = a.verify(sa, 5, [])["accept"][1]
    b.verify(sb, 5, [])
    x, y = a.verify(sa, best, [7, 8, 9]), b.verify_tree(sb, best, [7, 8, 9], [0, 1, 2])
    assert torch.equal(x["logits"], y["logits"]) and x["accept"] == y["accept"] and sa.length == sb.length
    assert torch.equal(x["scores"]["logprob"], y["scores"]["logprob"])
    for s, t in zip(_rows(a, sa, sa.length), _rows(b, sb, sb.length)):
        assert torch.equal(s, t)


def test_drawn_drafts_and_long_loops():
    """Steps of trees whose drafts are drawn from a draft distribution: lengths, pages and status stay consistent."""
    model = _model()
    seq = model.new_sequence()
    model.prefill(seq, list(range(60)))
    g = torch.Generator(device="cuda").manual_seed(3)
    last, total = 1, 60
    for step in range(12):
        q = torch.randn(4, 1000, generator=g, device="cuda")
        kids = torch.multinomial(torch.softmax(q[0].double() / 0.9, 0), 2, generator=g).tolist()
        deep = torch.multinomial(torch.softmax(q[1].double() / 0.9, 0), 1, generator=g).tolist()
        r = model.verify_tree(seq, last, kids + deep, [0, 0, 1], temperature=0.9, draft_logits=q)
        n, last = r["accept"]
        total += 1 + n
        assert seq.length == total and 0 <= last < 1000 and len(r["path"]) == n + 1
    model.block.attention.status()


def test_bad_trees_are_refused_before_anything_changes():
    model = _model()
    seq = model.new_sequence()
    model.prefill(seq, list(range(30)))
    for drafts, parents in (([1, 2], [0]), ([1, 2], [0, 2]), ([1], [-1]), ([1] * 64, [0] * 64)):
        with pytest.raises(MoEError, match="parents"):
            model.verify_tree(seq, 3, drafts, parents)
    assert seq.length == 30
    with pytest.raises(MoEError, match="longest"):
        seq.length = model.max_len - 1
        model.verify_tree(seq, 3, [1, 2], [0, 0])


def test_a_refused_step_keeps_no_node():
    """Numbers or draft rows of the wrong size: the sequence is as it was, and the next step gives what it would have given."""
    a, b = _model(), _model()
    sa, sb = a.new_sequence(), b.new_sequence()
    a.prefill(sa, list(range(50)))
    b.prefill(sb, list(range(50)))
    with pytest.raises(MoEError, match="uniforms"):
        a.verify_tree(sa, 3, [1, 2], [0, 0], uniforms=[0.5, 0.5])
    with pytest.raises(MoEError, match="draft_logits"):
        a.verify_tree(sa, 3, [1, 2], [0, 0], draft_logits=torch.zeros(2, 1000, device="cuda"))
    assert sa.length == 50
    x, y = (m.verify_tree(s, 3, [1, 2], [0, 0], uniforms=[0.3, 0.4, 0.5], temperature=0.7) for m, s in ((a, sa), (b, sb)))
    assert torch.equal(x["logits"], y["logits"]) and x["accept"] == y["accept"] and sa.length == sb.length
