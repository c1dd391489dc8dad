"""Answer one prompt several ways over one 8-bit paged cache.

A small random decoder (no trained weights) runs a ragged batch of prompts, forks each into
branches that share its pages, decodes every branch a token at a time, ends the branch that
does worst, renumbers the pages that are left and goes on.  Each layer of each step is the
same three calls: positions of the queries, quantising append of keys and values (keys turned
on the way), attention over the cache.

    python examples/branches.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from layer_wise_paged_gb300.cache import QuantCache, Rope, rotary  # noqa: E402


class Decoder:
    """Layers of grouped attention with a residual, then logits; bf16 weights from a seed."""

    def __init__(self, layers=3, heads=8, kv_heads=2, dim=128, width=512, vocab=1000, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g) / shape[0] ** 0.5).to(torch.bfloat16).cuda()

        self.layers, self.heads, self.kv_heads, self.dim, self.width = layers, heads, kv_heads, dim, width
        self.embed = weight(vocab, width) * vocab ** 0.5
        self.qkv = [weight(width, (heads + 2 * kv_heads) * dim) for _ in range(layers)]
        self.out = [weight(heads * dim, width) for _ in range(layers)]
        self.head = weight(width, vocab)
        self.rope = Rope.make(dim, base=10000.0)

    def step(self, cache, tokens, positions, starts, slots, max_new):
        """Logits [rows, vocab] of fresh tokens whose pages the cache has handed out; the last layer's q and
        attention too."""
        x = self.embed[tokens]
        h, n = self.heads, self.kv_heads
        for layer in range(self.layers):
            norm = torch.nn.functional.rms_norm(x.float(), (self.width,)).to(torch.bfloat16)
            rows = (norm @ self.qkv[layer]).view(-1, h + 2 * n, self.dim)  # q, k, v: parts of one tensor's rows
            q, k, v = rows[:, :h], rows[:, h:h + n], rows[:, h + n:]
            rotary(self.rope, positions, [(q, q)])
            cache.append(layer, k, v, starts, rope=self.rope, slots=slots)
            o = cache.attend(layer, q, starts, slots=slots, max_new=max_new)
            x = x + o.view(-1, h * self.dim) @ self.out[layer]
        return torch.nn.functional.rms_norm(x.float(), (self.width,)) @ self.head.float(), q, o


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(prompts=(37, 300, 1), branches=3, steps=12, block_tokens=16, code="e4m3", compact=True, watch=None):
    """Tokens [branches of all prompts][steps], ending branches dropped half-way; see the module's text.
    watch(cache, layer, slots, starts, q, out) is called after every step, if given."""
    model = Decoder()
    n_slots, pages = len(prompts) * branches, 64
    cache = QuantCache.empty(model.layers, model.kv_heads, model.dim, block_tokens, n_slots * pages, n_slots, pages,
                             code=code)

    def advance(slots, tokens, counts, first):
        """One step: counts[i] fresh tokens of slots[i], whose first stands at position first[i]."""
        starts = [0]
        for c in counts:
            starts.append(starts[-1] + c)
        s, st = _ints(slots), _ints(starts)
        cache.extend(s, _ints(counts))  # lengths, pages, and copies of partly filled pages that are shared
        cache.copy_pages()
        at = _ints([f + t for f, c in zip(first, counts) for t in range(c)])
        logits, q, out = model.step(cache, tokens, at, st, s, max(counts))
        if watch:
            watch(cache, model.layers - 1, s, st, q, out)
        return logits[st[1:].long() - 1]

    # the prompts, one ragged batch
    g = torch.Generator().manual_seed(1)
    tokens = torch.randint(0, model.embed.shape[0], (sum(prompts),), generator=g).cuda()
    slots = [i * branches for i in range(len(prompts))]
    logits = advance(slots, tokens, list(prompts), [0] * len(prompts))

    # branch b of a prompt starts with its b-th likeliest token
    children = [(p, p + b) for p in slots for b in range(1, branches)]
    if children:
        cache.fork(_ints([p for p, _ in children]), _ints([c for _, c in children]))
    live = list(range(n_slots))
    length = [prompts[s // branches] for s in live]
    tops = logits.topk(branches, dim=1)
    token, score = tops.indices.flatten(), tops.values.flatten().clone()
    said = [[] for _ in live]
    for step in range(steps):
        if step == steps // 2 and branches > 1:  # the worst branch of each prompt ends
            worst = score.view(len(prompts), -1).argmin(1).tolist()
            gone = [p * branches + w for p, w in enumerate(worst)]
            cache.free(_ints(gone))
            keep = [i for i, s in enumerate(live) if s not in gone]
            live, token, score = [live[i] for i in keep], token[keep], score[keep]
            if compact:
                cache.compact()
                cache.copy_pages()
        for s, t in zip(live, token.tolist()):
            said[s].append(t)
        logits = advance(live, token, [1] * len(live), [length[s] for s in live])
        for s in live:
            length[s] += 1
        best = logits.max(1)
        token, score = best.indices, score + best.values
    status = cache.status()
    if status != (0, 0):
        raise RuntimeError(f"the cache reports {status}")
    return said, cache


if __name__ == "__main__":
    answers, held = run()
    for number, answer in enumerate(answers):
        print(f"branch {number}: {answer}")
    live_pages = torch.nonzero(held.refs).flatten()
    print(f"{len(live_pages)} pages live, the highest numbered {int(live_pages.max())}; "
          f"{int((held.refs > 1).sum())} shared")
