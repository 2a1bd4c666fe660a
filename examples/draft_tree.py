"""Speculative decoding with drafted trees on a small random model: the package's operators in the order of a serving
loop.

Each round, for every request,
  1. a draft model grows a tree: ``spec_beam_select`` keeps the best continuations of a level's beams, and
     ``spec_beam_reorder`` brings the beams' states into their new order;
  2. the target runs all drafted tokens at once: ``spec_tree_attention`` reads the paged cache and each token's
     ancestors;
  3. ``spec_verify_greedy`` finds how far each of the tree's branches agrees with the target;
  4. ``spec_cache_commit`` writes the keys and values of the longest agreed branch to the cache;
  5. ``spec_attention_weights`` adds up what each cached token received, and when a cache is full,
     ``spec_cache_evict`` keeps the tokens of largest weight.

Run it with ``python examples/draft_tree.py`` on a GB300.  Without eviction the text is that of greedy decoding token
by token (``generate(..., drafts=False)``), in fewer rounds, up to ties within the rounding of bf16 activations.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_verification_23_gb300 as sv  # noqa: E402

DEV = "cuda"


class Target:
    """A few attention layers over token and place embeddings, with random weights."""

    def __init__(self, seed=0, vocab=1000, width=256, layers=2, heads=8, kv_heads=2, dim=64):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def w(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device=DEV) * scale / shape[0] ** 0.5).bfloat16()

        self.vocab, self.layers, self.heads, self.kv_heads, self.dim = vocab, layers, heads, kv_heads, dim
        self.embed = (torch.randn(vocab, width, generator=g, device=DEV)).bfloat16()
        self.place = (0.2 * torch.randn(4096, width, generator=g, device=DEV)).bfloat16()
        self.wq = [w(width, heads * dim) for _ in range(layers)]
        self.wk = [w(width, kv_heads * dim) for _ in range(layers)]
        self.wv = [w(width, kv_heads * dim) for _ in range(layers)]
        self.wo = [w(heads * dim, width, scale=0.7) for _ in range(layers)]
        self.head = w(width, vocab, scale=3.0)

    def run(self, tokens, places, cache, table, ctx, cu, nodes, mask):
        """Logits [n, vocab] of drafted tokens [n], and their keys, values, and the first layer's queries and lse."""
        x = self.embed[tokens] + self.place[places]
        ks, vs, first = [], [], None
        for i in range(self.layers):
            y = torch.nn.functional.rms_norm(x, x.shape[-1:])
            q = (y @ self.wq[i]).unflatten(-1, (self.heads, self.dim))
            k = (y @ self.wk[i]).unflatten(-1, (self.kv_heads, self.dim))
            v = (y @ self.wv[i]).unflatten(-1, (self.kv_heads, self.dim))
            args = sv.make_tree_args(q=q, k_new=k, v_new=v, cu_nodes=cu, max_nodes=nodes, tree_mask=mask, cache=cache,
                                     block_table=table, ctx_len=ctx, layer=i)
            out, lse, status = sv.spec_tree_attention(args)
            assert int(status.abs().max()) == 0
            first = (q, lse) if i == 0 else first
            x = x + out.flatten(1) @ self.wo[i]
            ks.append(k)
            vs.append(v)
        logits = torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head
        return logits, torch.stack(ks), torch.stack(vs), first

    def draft(self, tokens, places):
        """The draft model: the target without its attention."""
        x = self.embed[tokens] + self.place[places]
        return torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head


def grow(model, last, ctx, beams, depth):
    """Drafted trees of `beams` tokens a level under each request's last token (node 0).  Returns tokens [B, n], depths
    [n], ancestor bits [B, n], parents [B, n] and the last level's first node."""
    B = last.numel()
    tokens, masks, parents, depths = [last[:, None]], [torch.ones(B, 1, dtype=torch.int32, device=DEV)], [], [0]
    parents.append(torch.full((B, 1), -1, dtype=torch.int64, device=DEV))
    scores = torch.zeros(B, 1, device=DEV)
    node = torch.zeros(B, 1, dtype=torch.int32, device=DEV)      # the beams' nodes
    bits = masks[0].clone()                                       # and their ancestors
    for level in range(1, depth + 1):
        W = scores.shape[1]
        here = tokens[-1].flatten().long()
        logits = model.draft(here, (ctx[:, None] + (level - 1)).expand(B, W).flatten().long())
        scores, parent, token, status = sv.spec_beam_select(
            sv.make_beam_args(logits=logits, V=model.vocab, scores=scores, keep=beams))
        assert int(status.abs().max()) == 0
        above, seen = (torch.empty(B, beams, dtype=torch.int32, device=DEV) for _ in range(2))
        sv.spec_beam_reorder(sv.make_reorder_args(parents=parent, beams=W, states=[(node, above), (bits, seen)]))
        first = 1 + (level - 1) * beams
        node = torch.arange(first, first + beams, dtype=torch.int32, device=DEV).expand(B, beams).contiguous()
        bits = seen | (1 << node)
        tokens.append(token)
        masks.append(bits)
        parents.append(above.long())
        depths += [level] * beams
    return (torch.cat(tokens, 1), torch.tensor(depths, device=DEV), torch.cat(masks, 1), torch.cat(parents, 1),
            1 + (depth - 1) * beams)


def generate(seed=0, requests=3, rounds=20, beams=4, depth=3, page=16, drafts=True, keep=None, model=None):
    """Decodes `rounds` rounds greedily from one start token a request; `keep` bounds the caches by eviction.  Returns
    the requests' tokens and the caches' lengths."""
    model = model or Target(seed)
    B, most = requests, (rounds + 1) * (depth + 1) + page
    pages = -(-most // page)
    shape = (model.layers, 2 * B * pages, page, model.kv_heads, model.dim)
    k, v = (torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = sv.make_cache(k, v)
    free = torch.randperm(2 * B * pages, generator=torch.Generator().manual_seed(seed)).to(DEV, torch.int32)
    table, spare = free[:B * pages].view(B, pages).contiguous(), free[B * pages:].view(B, pages).contiguous()
    ctx = torch.zeros(B, dtype=torch.int32, device=DEV)
    place = torch.zeros(B, dtype=torch.int32, device=DEV)        # the last token's place in the text
    last = torch.arange(B, dtype=torch.int32, device=DEV)
    weights = torch.zeros(B, model.kv_heads, pages * page, device=DEV)
    text = [[int(t)] for t in last]
    for _ in range(rounds):
        if drafts:
            tokens, depths, masks, parents, leaf = grow(model, last, place, beams, depth)
        else:
            tokens, depths, leaf = last[:, None], torch.zeros(1, dtype=torch.int64, device=DEV), 0
            masks, parents = torch.ones_like(tokens), torch.full((B, 1), -1, dtype=torch.int64, device=DEV)
        n = tokens.shape[1]
        cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
        logits, k_new, v_new, (q, lse) = model.run(tokens.flatten().long(), (place[:, None] + depths).flatten().long(),
                                                   cache, table, ctx, cu, n, masks.flatten()[:, None].contiguous())
        # every branch from the root to a leaf, verified as a chain of drafts
        leaves = torch.arange(leaf, n, device=DEV).expand(B, -1)
        branch = [leaves]
        for _ in range(int(depths[-1])):
            branch.append(torch.gather(parents, 1, branch[-1]))
        branch = torch.stack(branch[::-1], 2)                     # [B, leaves, depth + 1] nodes
        L, D = branch.shape[1], branch.shape[2] - 1
        rows = logits.view(B, n, -1)[torch.arange(B, device=DEV)[:, None, None], branch].flatten(0, 2).contiguous()
        path_tokens = torch.gather(tokens, 1, branch.flatten(1)).view(B, L, D + 1).int()
        cu_draft = torch.arange(0, B * L * D + 1, D, dtype=torch.int32, device=DEV) if D else torch.zeros(
            B * L + 1, dtype=torch.int32, device=DEV)
        proposed = path_tokens[:, :, 1:].reshape(-1).contiguous()     # held: this argument block keeps no tensor
        out, accepted, status = sv.spec_verify_greedy(
            sv.make_args(target=rows, cu_draft=cu_draft, draft_tokens=proposed, V=model.vocab, max_k=D))
        assert int(status.abs().max()) == 0
        accepted, out = accepted.view(B, L), out.view(B, L, D + 1)
        best = accepted.argmax(1)
        count = (accepted.gather(1, best[:, None])[:, 0] + 1).int()   # nodes to commit: the root and what agreed
        path = branch[torch.arange(B, device=DEV), best].int().contiguous()
        new_len, status = sv.spec_cache_commit(
            sv.make_commit_args(k_new=k_new, v_new=v_new, cu_nodes=cu, path=path, path_len=count, cache=cache,
                                block_table=table, ctx_len=ctx))
        assert int(status.abs().max()) == 0
        said = out[torch.arange(B, device=DEV), best]
        for b, (m, toks) in enumerate(zip(count.tolist(), said.tolist())):
            text[b] += toks[:m]
        last = said.gather(1, count[:, None].long() - 1)[:, 0].contiguous()
        place, ctx = place + count, new_len
        # what the committed tokens' first layer paid attention to
        taken = (torch.arange(D + 1, device=DEV) < count[:, None])
        at = (torch.arange(B, device=DEV)[:, None] * n + path)[taken].long()
        cu_rows = torch.cat([torch.zeros(1, device=DEV), count.cumsum(0)]).int()
        weights, status = sv.spec_attention_weights(
            sv.make_weigh_args(q=q[at].contiguous(), lse=lse[at].contiguous(), cu_rows=cu_rows, max_rows=D + 1,
                               cache=cache, block_table=table, kv_len=ctx), weights)
        assert int(status.abs().max()) == 0
        if keep is not None and int(ctx.max()) > keep + page:
            # one selection a layer; here the first layer's weights serve all
            for layer in range(model.layers):
                index, kept, new_len, status = sv.spec_cache_evict(
                    sv.make_evict_args(weights=weights, kv_len=ctx, keep=keep, sink=2, recent=keep // 4, cache=cache,
                                       block_table=table, to_table=spare, layer=layer))
                assert int(status.abs().max()) == 0
            table, spare, ctx = spare, table, new_len
            weights = torch.nn.functional.pad(kept, (0, weights.shape[2] - keep)).contiguous()
    return text, ctx.tolist()


def shortfalls(model, text, page=16):
    """How far below the largest logit each token of a text (one request's, at most 256 tokens) is when the model reads
    the whole text as one chain of drafted tokens, and the largest size of a logit."""
    n = len(text) - 1
    t = torch.tensor(text, device=DEV)
    shape = (model.layers, 1, page, model.kv_heads, model.dim)
    cache = sv.make_cache(*(torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    none = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    logits = model.run(t[:n], torch.arange(n, device=DEV), cache, none, none[0], torch.tensor([0, n], dtype=torch.int32, device=DEV),
                       n, None)[0].float()
    return (logits.amax(1) - logits[torch.arange(n, device=DEV), t[1:]]).tolist(), float(logits.abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=30)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--depth", type=int, default=3)
    a = ap.parse_args()
    if a.beams * a.depth > 31:
        ap.error("a tree of at most 32 tokens here: --beams times --depth below 32")
    model = Target()
    text, lens = generate(rounds=a.rounds, requests=a.requests, beams=a.beams, depth=a.depth, model=model)
    for b, t in enumerate(text):
        print(f"request {b}: {len(t) - 1} tokens in {a.rounds} rounds, cache {lens[b]}: {t[:12]} ...")
    text, lens = generate(rounds=a.rounds, requests=a.requests, beams=a.beams, depth=a.depth, keep=32, model=model)
    print("with eviction to 32 tokens: caches", lens)


if __name__ == "__main__":
    main()
