"""One decoder block and a draft/verify step over it: the attention operators,
the MoE layer, the LM head, greedy acceptance and token scores as a serving
loop uses them together.

    block = synthetic_block(...)            # attention + MoE of one layer
    model = Decoder(embed, block, lm_head)  # (one layer: the loop is the same for more)
    model.prefill(seq, prompt)              # prompt tokens into the cache, in chunks
    model.verify(seq, last, drafts)         # the k+1 verify rows: accepted count, next token, scores

Projections are plain torch products (the library's operators take and return
the tensors between them).  Synthetic weights only.

    python -m block_quantized_moe_layer_gb300.decoder

runs a prompt and three verify steps of the pages' shapes ("Step-5 Preview
GGUF", "Model background" table: 64 query and 4 key/value heads of 192
channels, 64 of them rotated, a window of 512 in the sliding layers) and
prints what was accepted.
"""
from dataclasses import dataclass

import torch

from . import ACT_BF16, MOE_EINVAL, Attention, Layer, LmHead, MoEError, token_logprobs, verify_accept


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

    def forward(self, h, positions, slots, starts, lens, table, max_q, max_len):
        """h fp32 [T, H]: the new tokens of every sequence, in order."""
        at = self.attention
        T = h.shape[0]
        qkv = (rmsnorm(h) @ self.w_qkv).unflatten(1, (-1, at.head_dim))
        q, k, v = qkv.split([at.n_q_heads, at.n_kv_heads, at.n_kv_heads], 1)
        q = at.append(q, k, v, positions, slots, self.cache)
        o = at.forward(q, self.cache, starts, lens, table, max_q, max_len)
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

    def _run(self, seq, tokens):
        """Appends `tokens` (a host list) to the sequence; the block's output rows."""
        at, dev = self.block.attention, self.embed.device
        P, n, first = at.page_tokens, len(tokens), seq.length
        if first + n > self.max_len:
            raise MoEError(MOE_EINVAL, f"{first} + {n} tokens: the longest sequence has {self.max_len}")
        if first + n > (len(seq.pages) + len(self.free)) * P:
            raise MoEError(MOE_EINVAL, f"{first} + {n} tokens: {len(self.free)} pages of {P} are left")
        while len(seq.pages) * P < first + n:
            seq.pages.append(self.free.pop())
        pos = torch.arange(first, first + n, dtype=torch.int32)
        page = torch.tensor(seq.pages, dtype=torch.int32)
        slots = page[(pos // P).long()].long() * P + pos % P
        ids = torch.tensor(tokens, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        out = self.block.forward(self.embed[ids].float(), pos.to(dev), slots.to(dev), torch.tensor([0, n], **i32),
                                 torch.tensor([first + n], **i32), page.to(dev)[None], n, first + n)
        seq.length = first + n
        return out

    def prefill(self, seq, prompt):
        """The prompt's tokens into the cache, chunk by chunk."""
        for i in range(0, len(prompt), self.chunk):
            self._run(seq, prompt[i:i + self.chunk])

    def verify(self, seq, last, drafts, n_top=4):
        """One verify step of [last] + drafts (at most 7): a dict of the rows'
        logits, accept [n, next] (``verify_accept``), and the scores of the
        tokens that were checked (``token_logprobs``).  The rows of rejected
        drafts leave the sequence again (their slots are written over)."""
        h = self._run(seq, [last] + list(drafts))
        logits = torch.cat([self.lm.forward(h[i:i + self.lm.T_max].to(torch.bfloat16)) for i in range(0, h.shape[0], self.lm.T_max)])
        ids = torch.tensor(drafts, dtype=torch.int32, device=h.device)
        accept = verify_accept(ids, logits)
        n, nxt = accept.tolist()
        checked = torch.tensor(list(drafts[:n]) + [nxt], dtype=torch.int32, device=h.device)
        seq.length -= len(drafts) - n
        return dict(logits=logits, accept=[n, nxt], hidden=h, scores=token_logprobs(logits[:n + 1], checked, n_top))


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
    model.block.attention.status()


if __name__ == "__main__":
    main()
