"""One decoder block and a draft/verify step over it: the attention operators,
the MoE layer, the LM head, acceptance (greedy of a chain of drafts, sampled of
a tree of them) and token scores as a serving loop uses them together.

    block = synthetic_block(...)            # attention + MoE of one layer
    model = Decoder(embed, block, lm_head)  # (one layer: the loop is the same for more)
    model.prefill(seq, prompt)              # prompt tokens into the cache, in chunks
    model.verify(seq, last, drafts)         # the k+1 verify rows: accepted count, next token, scores
    model.verify_tree(seq, last, drafts, parents, temperature=0.8)  # the same of a tree, drawn at a temperature

Projections are plain torch products (the library's operators take and return
the tensors between them).  Synthetic weights only.

    python -m block_quantized_moe_layer_gb300.decoder

runs a prompt and three verify steps, and three of trees, of the pages' shapes ("Step-5 Preview
GGUF", "Model background" table: 64 query and 4 key/value heads of 192
channels, 64 of them rotated, a window of 512 in the sliding layers) and
prints what was accepted.
"""
from dataclasses import dataclass

import torch

from . import ACT_BF16, MOE_EINVAL, Attention, Layer, LmHead, MoEError, token_logprobs, verify_accept, verify_sample


def rmsnorm(h, eps=1e-6):
    """bf16 rows of fp32 rows h (weight 1)."""
    return (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps)).to(torch.bfloat16)


@dataclass
class Sequence:
    """One sequence's place in the cache: its pages and how many tokens they hold."""
    pages: list
    length: int = 0


class Block:
    """One pre-norm decoder block: h += Wo attention(rmsnorm h), h += MoE(rmsnorm h)."""

    def __init__(self, attention: Attention, w_qkv, w_out, moe: Layer):
        self.attention, self.w_qkv, self.w_out, self.moe = attention, w_qkv, w_out, moe
        self.cache = attention.pages(w_qkv.device)

    def forward(self, h, positions, slots, starts, lens, table, max_q, max_len, parents=None):
        """h fp32 [T, H]: the new tokens of every sequence, in order, or with
        parents (int32 [T]) the nodes of their trees."""
        at = self.attention
        T = h.shape[0]
        qkv = (rmsnorm(h) @ self.w_qkv).unflatten(1, (-1, at.head_dim))
        q, k, v = qkv.split([at.n_q_heads, at.n_kv_heads, at.n_kv_heads], 1)
        q = at.append(q, k, v, positions, slots, self.cache)
        o = at.forward(q, self.cache, starts, lens, table, max_q, max_len, parents=parents)
        h = h + (o.view(T, -1) @ self.w_out).float()
        return h + self.moe.forward(rmsnorm(h)).float()


class Decoder:
    """An embedding, one block and the LM head over a paged cache.  ``chunk``:
    prompt tokens of one prefill call."""

    def __init__(self, embed, block: Block, lm: LmHead, max_len, chunk=1024):
        self.embed, self.block, self.lm, self.max_len, self.chunk = embed, block, lm, max_len, chunk
        self.free = list(range(block.attention.n_pages))[::-1]

    def new_sequence(self):
        return Sequence([])

    def _run(self, seq, tokens, parents=None):
        """Appends `tokens` (a host list), or with `parents` the nodes of a tree, to the sequence; the block's output rows."""
        at, dev = self.block.attention, self.embed.device
        P, n, first = at.page_tokens, len(tokens), seq.length
        if first + n > self.max_len:
            raise MoEError(MOE_EINVAL, f"{first} + {n} tokens: the longest sequence has {self.max_len}")
        if first + n > (len(seq.pages) + len(self.free)) * P:
            raise MoEError(MOE_EINVAL, f"{first} + {n} tokens: {len(self.free)} pages of {P} are left")
        while len(seq.pages) * P < first + n:
            seq.pages.append(self.free.pop())
        place = torch.arange(first, first + n, dtype=torch.int32)
        page = torch.tensor(seq.pages, dtype=torch.int32)
        slots = page[(place // P).long()].long() * P + place % P
        pos = place
        if parents is not None:  # a node stands behind its parent, wherever its row lies
            depth = []
            for p in parents:
                depth.append(depth[p] + 1 if p >= 0 else 0)
            pos = first + torch.tensor(depth, dtype=torch.int32)
        ids = torch.tensor(tokens, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        out = self.block.forward(self.embed[ids].float(), pos.to(dev), slots.to(dev), torch.tensor([0, n], **i32),
                                 torch.tensor([first + n], **i32), page.to(dev)[None], n, first + n,
                                 None if parents is None else torch.tensor(parents, **i32))
        seq.length = first + n
        return out

    def prefill(self, seq, prompt):
        """The prompt's tokens into the cache, chunk by chunk."""
        for i in range(0, len(prompt), self.chunk):
            self._run(seq, prompt[i:i + self.chunk])

    def _logits(self, h):
        T = self.lm.T_max
        return torch.cat([self.lm.forward(h[i:i + T].to(torch.bfloat16)) for i in range(0, h.shape[0], T)])

    def verify(self, seq, last, drafts, n_top=4):
        """One verify step of [last] + drafts (at most 7): a dict of the rows'
        logits, accept [n, next] (``verify_accept``), and the scores of the
        tokens that were checked (``token_logprobs``).  The rows of rejected
        drafts leave the sequence again (their slots are written over)."""
        h = self._run(seq, [last] + list(drafts))
        logits = self._logits(h)
        ids = torch.tensor(drafts, dtype=torch.int32, device=h.device)
        accept = verify_accept(ids, logits)
        n, nxt = accept.tolist()
        checked = torch.tensor(list(drafts[:n]) + [nxt], dtype=torch.int32, device=h.device)
        seq.length -= len(drafts) - n
        return dict(logits=logits, accept=[n, nxt], hidden=h, scores=token_logprobs(logits[:n + 1], checked, n_top))


    def verify_tree(self, seq, last, drafts, parents, uniforms=None, temperature=0.0, draft_logits=None, n_top=4):
        """One verify step of a tree: node 0 is `last`, node i the draft
        drafts[i - 1] behind node parents[i - 1] (at most 63 drafts, a parent
        before its children).  `uniforms`: len(drafts) + 1 numbers in [0, 1)
        (:func:`verify_sample`; default: drawn here); `draft_logits` [nodes, V]
        fp32, or None for drafts chosen without chance.  A dict as
        :meth:`verify` returns, with `path`, the nodes that were kept; the
        others' rows leave the sequence."""
        at, dev = self.block.attention, self.embed.device
        n, tree = len(drafts) + 1, [-1] + list(parents)
        if len(tree) != n or any(not 0 <= p < i for i, p in enumerate(tree[1:], 1)) or n > 64:
            raise MoEError(MOE_EINVAL, f"{len(drafts)} drafts with parents {list(parents)}: an earlier node each, at most 63")
        first = seq.length
        h = self._run(seq, [last] + list(drafts), tree)
        seq.length = first  # (until the nodes that stay are known: a call that is refused on the way leaves none)
        logits = self._logits(h)
        i32 = dict(dtype=torch.int32, device=dev)
        nodes, lens = torch.tensor([0, n], **i32), torch.tensor([first + n], **i32)
        numbers = torch.rand(n, device=dev) if uniforms is None else torch.as_tensor(uniforms, dtype=torch.float32, device=dev)
        r = verify_sample(logits, torch.tensor([last] + list(drafts), **i32), torch.tensor(tree, **i32), nodes, numbers, n,
                          draft_logits=draft_logits, temperature=torch.tensor([temperature], dtype=torch.float32, device=dev))
        table = torch.tensor([seq.pages], **i32)
        kept = at.commit(self.block.cache, nodes, lens, table, r["path"], first + n)
        length, accepted, nxt, *path = torch.cat([kept, r["n_accepted"], r["next"], r["path"][0]]).tolist()
        path = path[:accepted + 1]
        seq.length = length
        checked = torch.tensor([drafts[i - 1] for i in path[1:]] + [nxt], **i32)
        scores = token_logprobs(logits[torch.tensor(path, device=dev)], checked, n_top)
        return dict(logits=logits, accept=[accepted, nxt], path=path, hidden=h, scores=scores)


def synthetic_block(workload, n_q_heads, n_kv_heads, head_dim, rot_dim, page_tokens, n_pages, max_len, T_max, window=0, seed=0,
                    device="cuda"):
    """A block of synthetic weights around the MoE layer of `workload` (:mod:`.synth`)."""
    from .workloads import synthetic_layer
    g = torch.Generator(device=device).manual_seed(seed)
    H, width = workload.H, head_dim * n_q_heads

    def w(rows, cols):
        return (torch.randn(rows, cols, generator=g, device=device) / rows ** 0.5).to(torch.bfloat16)

    at = Attention(n_q_heads, n_kv_heads, head_dim, page_tokens, n_pages, T_max, 1, max_len, rot_dim=rot_dim,
                   q_norm=torch.ones(head_dim, device=device), k_norm=torch.ones(head_dim, device=device), window=window)
    moe, _ = synthetic_layer(workload, ACT_BF16, T_max=T_max, device=device)
    return Block(at, w(H, width + 2 * head_dim * n_kv_heads), w(width, H), moe)


def synthetic_decoder(workload, vocab, prompt_max, **block):
    """A Decoder of synthetic weights; `block`: synthetic_block's arguments."""
    from . import FMT_Q8_0, quantize
    dev = block.get("device", "cuda")
    g = torch.Generator(device=dev).manual_seed(block.get("seed", 0) + 1)
    b = synthetic_block(workload, max_len=prompt_max + 64, T_max=min(1024, prompt_max),
                        n_pages=-(-(prompt_max + 64) // block["page_tokens"]) + 1, **block)
    embed = torch.randn(vocab, workload.H, generator=g, device=dev).to(torch.bfloat16)
    head = quantize(FMT_Q8_0, torch.randn(vocab, workload.H, generator=g, device=dev) * 0.02)
    return Decoder(embed, b, LmHead(head, vocab, workload.H, 8, ACT_BF16), prompt_max + 64, chunk=min(1024, prompt_max))


def main():
    from dataclasses import replace

    from . import synth
    w = replace(synth.WORKLOADS["verify_mixed"], E=32)  # 32 of the 352 experts, to start quickly
    model = synthetic_decoder(w, 32768, 4000, n_q_heads=64, n_kv_heads=4, head_dim=192, rot_dim=64, page_tokens=64, window=512)
    seq = model.new_sequence()
    model.prefill(seq, torch.randint(32768, (3500,)).tolist())
    last, drafts = 7, [1, 2, 3]
    for _ in range(3):
        r = model.verify(seq, last, drafts)
        n, last = r["accept"]
        print(f"{seq.length} tokens, accepted {n}, next {last}, log probabilities "
              f"{[round(v, 3) for v in r['scores']['logprob'].tolist()]}, entropies {[round(v, 3) for v in r['scores']['entropy'].tolist()]}")
        # the next drafts: the target's own choice after `last`, twice right and once wrong
        ahead = model._run(seq, [last])
        seq.length -= 1
        best = int(model.lm.forward(ahead.to(torch.bfloat16))[0].argmax())
        drafts = [best, (best + 1) % 32768, 5]
    # trees: two candidates for the next token, two behind the first, one behind the second
    for _ in range(3):
        ahead = model._run(seq, [last])
        seq.length -= 1
        first, second = model._logits(ahead)[0].topk(2).indices.tolist()
        r = model.verify_tree(seq, last, [first, second, 11, 12, 13], [0, 0, 1, 1, 2], temperature=0.8)
        n, last = r["accept"]
        print(f"{seq.length} tokens, accepted {n} (nodes {r['path']}), next {last}, log probabilities "
              f"{[round(v, 3) for v in r['scores']['logprob'].tolist()]}")
    model.block.attention.status()


if __name__ == "__main__":
    main()
