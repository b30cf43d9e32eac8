"""The attention operators, the MoE layer, the LM head, acceptance and scores
run together as a serving loop does."""
from dataclasses import replace

import numpy as np
import pytest
import torch

from block_quantized_moe_layer_gb300 import MoEError, decoder, synth
from oracle import accept as oacc
from oracle import attn as oa

pytestmark = pytest.mark.gpu


def _model(window=0):
    w = replace(synth.WORKLOADS["tiny"], H=512, I=128, I_shared=128)
    return decoder.synthetic_decoder(w, 1000, 300, n_q_heads=8, n_kv_heads=2, head_dim=64, rot_dim=32, page_tokens=16, window=window)


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("window", [0, 40])
def test_prefill_and_verify_steps(window):
    model = _model(window)
    at = model.block.attention
    rng = np.random.default_rng(0)
    prompt = rng.integers(0, 1000, 200).tolist()
    seq = model.new_sequence()
    model.prefill(seq, prompt)
    assert seq.length == 200 and len(seq.pages) == 13
    # the attention of a verify step is the oracle's over what the cache holds
    seen = {}
    forward = at.forward
    at.forward = lambda q, *a, **k: seen.setdefault("o", forward(seen.setdefault("q", q.clone()), *a, **k))
    r = model.verify(seq, 3, [4, 5, 6])
    del at.forward
    j = torch.arange(204, device="cuda")
    slots = torch.tensor(seq.pages, device="cuda")[j // 16] * 16 + j % 16
    keys, values = at.read(slots, model.block.cache)
    want, _, mag = oa.attention(_np(seen["q"]), _np(keys), _np(values), 4, window)
    # a rounding of the output (2^-8), of the weights (2^-11) and of exponentials and sums (2^-17 here)
    assert (np.abs(_np(seen["o"]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mag).all()
    # acceptance and scores are the oracles' on the step's logits
    logits = r["logits"].cpu().numpy()
    n, nxt, _ = oacc.greedy_accept([4, 5, 6], logits)
    assert r["accept"] == [n, nxt] and seq.length == 201 + n
    lp, en, ids, tl = oa.scores(logits[:n + 1], ([4, 5, 6][:n] + [nxt]), 4)
    assert np.allclose(_np(r["scores"]["logprob"]), lp, atol=1e-5) and np.allclose(_np(r["scores"]["entropy"]), en, atol=1e-4)
    assert np.array_equal(r["scores"]["top_ids"].cpu().numpy(), ids) and (ids[:, 0] == ([4, 5, 6][:n] + [nxt])).all()
    at.status()


def test_verify_rows_equal_the_same_tokens_one_by_one_up_to_rounding():
    """Verifying k+1 tokens at once gives the logits of decoding them singly,
    within the bf16 roundings of the block (other kernels, other sums)."""
    prompt = list(range(100, 200))
    a, b = _model(), _model()
    sa, sb = a.new_sequence(), b.new_sequence()
    a.prefill(sa, prompt)
    b.prefill(sb, prompt)
    many = a._run(sa, [1, 2, 3, 4])
    single = torch.cat([b._run(sb, [t]) for t in (1, 2, 3, 4)])
    # h is a sum of an embedding row (norm about sqrt H) and two bf16 products of
    # about its size: each of their three bf16 tensors is off by 2^-8 at most
    scale = many.norm(dim=1, keepdim=True)
    assert ((many - single).norm(dim=1, keepdim=True) <= 6 * 2.0 ** -8 * scale).all()


def test_rejected_drafts_leave_no_trace():
    model = _model()
    seq = model.new_sequence()
    model.prefill(seq, list(range(50)))
    best = int(model.verify(seq, 9, [])["accept"][1])
    seq.length -= 1
    wrong = (best + 1) % 1000
    r = model.verify(seq, 9, [wrong, 1, 2])
    assert r["accept"] == [0, best] and seq.length == 51
    once = model.verify(seq, best, [7])["logits"]
    fresh = model.new_sequence()
    model.free = [p for p in range(model.block.attention.n_pages) if p not in seq.pages]
    model.prefill(fresh, list(range(50)))
    model._run(fresh, [9])
    again = model.verify(fresh, best, [7])["logits"]
    assert torch.allclose(once, again, rtol=0, atol=3 * 2.0 ** -8 * float(once.abs().max()))


def test_a_step_that_does_not_fit_is_refused_before_anything_changes():
    model = _model()
    seq = model.new_sequence()
    model.prefill(seq, list(range(100)))
    pages, free = list(seq.pages), list(model.free)
    with pytest.raises(MoEError, match="longest"):
        model._run(seq, [1] * (model.max_len - 100 + 1))
    assert seq.length == 100 and seq.pages == pages and model.free == free
    model.free = model.free[:2]
    with pytest.raises(MoEError, match="pages"):
        model._run(seq, [1] * 60)
    assert seq.length == 100 and seq.pages == pages and len(model.free) == 2
    model._run(seq, [1] * 20)  # what fits still runs
    assert seq.length == 120
    model.block.attention.status()
