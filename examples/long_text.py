"""Speculative decoding of long texts: layers with a sliding window over a 16-bit cache whose old pages are given back,
between layers that see everything, over a cache in 8 bits.

Each round, for every request,
  1. a draft model grows a tree (see ``draft_tree``);
  2. the target runs all drafted tokens at once.  In every layer ``spec_norm_rotate`` norms the queries and keys and
     rotates them to their places in the text; even layers attend through ``spec_window_attention``, odd ones through
     ``spec_cache8_attention``;
  3. ``spec_verify_greedy`` finds the longest branch that agrees with the target;
  4. ``spec_cache_commit`` and ``spec_cache8_commit`` write its keys and values to the two caches;
  5. pages of the windowed layers that no later token sees are freed.

Run it with ``python examples/long_text.py`` on a GB300.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from draft_tree import DEV, Target, agree, grow, sv  # noqa: E402


class LongTarget(Target):
    """The target with norms and rotations of queries and keys in place of place embeddings' work in attention."""

    def __init__(self, window=24, sinks=2, **kw):
        super().__init__(**kw)
        self.window, self.sinks = window, sinks
        self.q_weight, self.k_weight = (torch.full((self.dim,), s, device=DEV).bfloat16() for s in (1.5, 1.0))
        self.inv_freq = (1e4 ** (-torch.arange(0, self.dim, 2, device=DEV) / self.dim)).float()

    def run(self, tokens, places, recent, whole, table, ctx, cu, nodes, mask):
        """Logits [n, vocab] of drafted tokens [n], and their keys and values [layers, n, heads, dim].  `recent` and
        `whole` are the windowed layers' cache and the others'; `table` a pair of block tables."""
        x = self.embed[tokens] + self.place[places]
        at = places.int()
        H, K = self.heads, self.kv_heads
        ks, vs = [], []
        for i in range(self.layers):
            y = torch.nn.functional.rms_norm(x, x.shape[-1:])
            q = (y @ self.wq[i]).unflatten(-1, (H, self.dim))
            k = (y @ self.wk[i]).unflatten(-1, (K, self.dim))
            v = (y @ self.wv[i]).unflatten(-1, (K, self.dim))
            sv.spec_norm_rotate(sv.make_rotate_args(q=q, k=k, positions=at, inv_freq=self.inv_freq,
                                                    q_weight=self.q_weight, k_weight=self.k_weight), out_q=q, out_k=k)
            drafted = dict(q=q, k_new=k, v_new=v, cu_nodes=cu, max_nodes=nodes, tree_mask=mask, ctx_len=ctx, layer=i // 2)
            if i % 2 == 0:
                out, _, status = sv.spec_window_attention(sv.make_window_args(
                    **drafted, cache=recent, block_table=table[0], window=self.window, sinks=self.sinks))
            else:
                out, _, status = sv.spec_cache8_attention(sv.make_cache8_args(**drafted, cache=whole, block_table=table[1]))
            assert int(status.abs().max()) == 0
            x = x + out.flatten(1) @ self.wo[i]
            ks.append(k)
            vs.append(v)
        logits = torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head
        return logits, torch.stack(ks), torch.stack(vs)


def generate(seed=0, requests=3, rounds=30, beams=4, depth=3, page=16, block=16, model=None):
    """Decodes `rounds` rounds greedily from one start token a request.  Returns the requests' tokens, the caches'
    lengths and the pages that the windowed layers hold at the end."""
    model = model or LongTarget(seed=seed, layers=4)
    B, pages = requests, -(-(rounds + 1) * (depth + 1) // page)
    heads, dim, half = model.kv_heads, model.dim, model.layers // 2
    recent = sv.make_cache(*(torch.empty(half, B * pages, page, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    whole = sv.make_cache8(*(torch.empty(half, B * pages, page, heads, dim, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)),
                           *(torch.empty(half, B * pages, page // block, heads, device=DEV) for _ in range(2)))
    g = torch.Generator().manual_seed(seed)
    table = [torch.randperm(B * pages, generator=g).to(DEV, torch.int32).view(B, pages).contiguous() for _ in range(2)]
    ctx = torch.zeros(B, dtype=torch.int32, device=DEV)
    last = torch.arange(B, dtype=torch.int32, device=DEV)
    text = [[int(t)] for t in last]
    first_slot = torch.arange(pages, device=DEV) * page
    for _ in range(rounds):
        tokens, depths, masks, parents, leaf = grow(model, last, ctx, beams, depth)
        n = tokens.shape[1]
        cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
        logits, k_new, v_new = model.run(tokens.flatten().long(), (ctx[:, None] + depths).flatten().long(), recent,
                                         whole, table, ctx, cu, n, masks.flatten()[:, None].contiguous())
        path, count, said = agree(model, logits, tokens, depths, parents, leaf)
        commit = dict(cu_nodes=cu, path=path, path_len=count, ctx_len=ctx)
        new_len, status = sv.spec_cache_commit(sv.make_commit_args(
            k_new=k_new[0::2], v_new=v_new[0::2], cache=recent, block_table=table[0], **commit))
        assert int(status.abs().max()) == 0
        ctx, status = sv.spec_cache8_commit(sv.make_cache8_commit_args(
            k_new=k_new[1::2], v_new=v_new[1::2], cache=whole, block_table=table[1], **commit))
        assert int(status.abs().max()) == 0 and torch.equal(ctx, new_len)
        for b, (m, toks) in enumerate(zip(count.tolist(), said.tolist())):
            text[b] += toks[:m]
        last = said.gather(1, count[:, None].long() - 1)[:, 0].contiguous()
        # the next token sees the sinks and, itself among them, the last `window`: pages that end before both are free
        old = (first_slot >= model.sinks) & (first_slot + page <= ctx[:, None] - model.window)
        table[0] = torch.where(old, -1, table[0])
    return text, ctx.tolist(), (table[0] >= 0).sum(1).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=60)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--depth", type=int, default=3)
    a = ap.parse_args()
    if a.beams * a.depth > 31:
        ap.error("a tree of at most 32 tokens here: --beams times --depth below 32")
    text, lens, held = generate(rounds=a.rounds, requests=a.requests, beams=a.beams, depth=a.depth)
    for t, n, h in zip(text, lens, held):
        print(f"{n} tokens in {a.rounds} rounds, {h} pages for the windowed layers:", *t[:12], "...")


if __name__ == "__main__":
    main()
