"""Measured cases of the operators beside the drafted tree: norms of queries and keys with the position rotation, tree
attention with a sliding window and sinks, tree attention over a cache held in 8 bits with a scale for each block of
tokens and head, and commitment of the accepted path (or a prompt) to such a cache.

Each case is one call as a serving loop makes it, on the inputs that such a loop has in hand.  `own` false computes the
plain form, elementary torch operations in 32 bits (64 for the angles of far positions); `own` true makes the package's
calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the drafter's own step, one token of one request: 14 heads in 2 groups of 64
        dict(name="rotate one token", op="rotate", rows=1, heads=14, kv_heads=2, dim=64, rot=64, pairs="halves",
             far=4096, dtype="bf16"),
        # a chunk of prompts through the target's projections: 28 heads in 4 groups of 128, far positions
        dict(name="rotate a prompt", op="rotate", rows=16384, heads=28, kv_heads=4, dim=128, rot=128, pairs="halves",
             far=131072, dtype="bf16"),
        # one token of one long chat with a window of 1024
        dict(name="window one token", op="window", batch=1, nodes=1, ragged=False, chain=True, heads=14, kv_heads=2,
             dim=64, ctx_lo=5001, ctx_hi=5001, page=16, window=1024, sinks=4, dtype="bf16"),
        # the verify step of 64 requests, 8 drafts and the last token each, most of them past their window
        dict(name="window chains", op="window", batch=64, nodes=9, ragged=True, chain=True, heads=28, kv_heads=4,
             dim=128, ctx_lo=257, ctx_hi=16384, page=16, window=4096, sinks=4, dtype="bf16"),
        # trees of up to 64 drafted tokens with a short window, half precision, large pages
        dict(name="window trees", op="window", batch=16, nodes=64, ragged=True, chain=False, heads=32, kv_heads=8,
             dim=128, ctx_lo=1024, ctx_hi=32768, page=64, window=2000, sinks=64, dtype="fp16"),
        # one token of a small draft model over an 8-bit cache
        dict(name="attend8 one token", op="attend8", batch=1, nodes=1, ragged=False, chain=True, heads=14, kv_heads=2,
             dim=64, ctx_lo=1001, ctx_hi=1001, page=16, block=16, window=0, sinks=0, dtype="bf16"),
        # the verify step of 64 ragged requests, a scale for each page
        dict(name="attend8 chains", op="attend8", batch=64, nodes=9, ragged=True, chain=True, heads=28, kv_heads=4,
             dim=128, ctx_lo=257, ctx_hi=8192, page=16, block=16, window=0, sinks=0, dtype="bf16"),
        # trees of up to 64 drafted tokens, half precision, large pages with four scales each
        dict(name="attend8 trees", op="attend8", batch=16, nodes=64, ragged=True, chain=False, heads=32, kv_heads=8,
             dim=128, ctx_lo=1024, ctx_hi=16384, page=64, block=16, window=0, sinks=0, dtype="fp16"),
        # two documents of up to 128 K tokens with a tree of 32: what an 8-bit cache is for
        dict(name="attend8 long", op="attend8", batch=2, nodes=32, ragged=False, chain=False, heads=16, kv_heads=8,
             dim=128, ctx_lo=100003, ctx_hi=131072, page=32, block=32, window=0, sinks=0, dtype="bf16"),
        # one request's accepted path written to every layer of the draft model's cache
        dict(name="commit8 one request", op="commit8", layers=24, batch=1, nodes=9, ragged=False, prompt=False,
             kv_heads=2, dim=64, ctx_lo=777, ctx_hi=777, page=16, block=16, dtype="bf16"),
        # 64 requests' paths, all 28 layers of the target's cache
        dict(name="commit8 a batch", op="commit8", layers=28, batch=64, nodes=33, ragged=True, prompt=False,
             kv_heads=4, dim=128, ctx_lo=100, ctx_hi=1000, page=16, block=16, dtype="bf16"),
        # prompts of up to 4096 tokens behind a shared system text, large pages
        dict(name="commit8 prompts", op="commit8", layers=16, batch=8, nodes=4096, ragged=True, prompt=True,
             kv_heads=8, dim=128, ctx_lo=0, ctx_hi=500, page=64, block=64, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "window", "window", "attend8", "attend8", "attend8", "commit8"])
    limit = [work(c) for c in listed() if c["op"] == op]
    most = {k: max(w[k] for w in limit) for k in ("bytes", "flops")}
    while True:
        kv = rng.choice([1, 2, 4, 8])
        c = dict(op=op, kv_heads=kv, dim=rng.choice([64, 128]), dtype=rng.choice(["bf16", "fp16"]))
        if op == "rotate":
            c.update(rows=_log(rng, 1, 16384), heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8]))
            c.update(rot=rng.choice([c["dim"], c["dim"] // 2]), pairs=rng.choice(["halves", "neighbours"]))
            c.update(far=_log(rng, 256, 1 << 20))
        else:
            c.update(batch=_log(rng, 1, 64), page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.5)
            c["block"] = rng.choice([x for x in (16, 32, 64, 128) if x <= c["page"]])
        if op in ("window", "attend8"):
            hi = _log(rng, 64, 131072)
            c.update(nodes=_log(rng, 1, 64), heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8]), chain=rng.random() < 0.4)
            c.update(ctx_lo=rng.choice([0, hi // 8, hi]), ctx_hi=hi, window=0, sinks=0)
            if op == "window" or rng.random() < 0.25:
                c.update(window=_log(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 16, 64, 130]))
            if op == "window":
                del c["block"]
        elif op == "commit8":
            c["prompt"] = rng.random() < 0.4
            hi = _log(rng, 16, 4096)
            c.update(layers=_log(rng, 1, 32), nodes=_log(rng, 1, 4096 if c["prompt"] else 64), ctx_lo=hi // 2, ctx_hi=hi)
        w = work(c)
        if all(w[k] <= most[k] for k in most) and _plain_bytes(c) <= 8 << 30:
            return c


def _plain_bytes(c):
    """What the plain form and the caches hold at once, roughly."""
    if c["op"] in ("window", "attend8"):
        keys = min(c["ctx_hi"], c["window"] + c["sinks"]) if c["window"] else c["ctx_hi"]
        held = c["batch"] * c["ctx_hi"] * c["kv_heads"] * c["dim"] * 4
        return held + c["batch"] * (keys + c["nodes"]) * 4 * (2 * c["kv_heads"] * c["dim"] + 3 * c["heads"] * c["nodes"])
    if c["op"] == "commit8":
        return c["layers"] * c["batch"] * (c["ctx_hi"] + 3 * c["nodes"]) * c["kv_heads"] * c["dim"] * 8
    return 0


def _lengths(n, lo, hi):
    """n whole numbers of lo..hi, ragged and always the same ones; the last is hi."""
    return [lo + ((i * 2654435761 + 1013904223) % (1 << 32)) * (hi - lo + 1) // (1 << 32) for i in range(n - 1)] + [hi]


def _counts(c, key):
    return _lengths(c["batch"], max(1, c[key] // 2) if c["ragged"] else c[key], c[key])


def _accepted(c):
    """Tokens that are committed: half of a drafted tree at most, a prompt whole."""
    return [n if c["prompt"] else max(1, n // 2) for n in _counts(c, "nodes")]


def work(c):
    if c["op"] == "rotate":
        values = c["rows"] * (c["heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": 4 * values + 4 * c["rows"], "flops": 8 * values}
    if c["op"] == "commit8":
        m, ctx = _accepted(c), _lengths(c["batch"], c["ctx_lo"], c["ctx_hi"])
        blocks = sum((a + x - 1) // c["block"] - a // c["block"] + 1 for a, x in zip(ctx, m))
        heads = c["layers"] * c["kv_heads"]
        return {"bytes": heads * (sum(m) * c["dim"] * 2 * 3 + blocks * 8), "flops": heads * sum(m) * c["dim"] * 4}
    ctx, n = _lengths(c["batch"], c["ctx_lo"], c["ctx_hi"]), _counts(c, "nodes")
    keys = [min(a, c["window"] + c["sinks"]) if c["window"] else a for a in ctx]
    pairs = sum(a * b for a, b in zip(keys, n)) + sum(n)  # a drafted token sees itself at least
    per = 2 if c["op"] == "window" else 1 + 4 / (c["block"] * c["dim"])  # bytes of a cached channel
    kv = (sum(keys) * per + sum(n) * 2) * c["kv_heads"] * c["dim"] * 2
    return {"bytes": int(kv + sum(n) * c["heads"] * (4 * c["dim"] + 4)), "flops": 4 * c["dim"] * c["heads"] * pairs}


# ------------------------------------------------------------------ the inputs

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cu(counts):
    return _i32(np.concatenate([[0], np.cumsum(counts)]).tolist())


def _table(rng, lens, page):
    """A block table of scattered pages for these lengths, and the number of pages."""
    need = [-(-n // page) for n in lens]
    ids = rng.permutation(sum(need))
    width, at = max(1, max(need)), 0
    table = np.zeros((len(lens), width), dtype=np.int32)
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(table).to(DEV), max(1, sum(need))


def _tree_masks(rng, counts, words):
    """Ancestor bits (itself among them) of drafted trees: a node's parent is one of the eight before it."""
    rows = []
    for n in counts:
        seen = []
        for i in range(n):
            mine = 1 << i
            if i:
                mine |= seen[rng.randint(max(0, i - 8), i)]
            seen.append(mine)
        rows += [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in seen]
    return torch.from_numpy(np.array(rows, dtype=np.uint32).view(np.int32)).to(DEV)


def prepare(case, seed):
    c = case
    rng = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape, dtype=t, scale=1.0):
        x = torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)
        return x.mul_(scale) if scale != 1.0 else x

    def held8(*shape):
        """An 8-bit cache [..., pages, page, heads, dim] of normal values and its scales: a block's largest value takes
        its scale near 448, and blocks differ in size."""
        x = normal(*shape, dtype=torch.float16, scale=90.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        sc = normal(*shape[:-3], c["page"] // c["block"], shape[-2], dtype=torch.float32, scale=0.3).exp_().mul_(1 / 90)
        return x, sc

    s = dict(c)
    if c["op"] == "rotate":
        # queries, keys and values of one projection, side by side
        s["qkv"] = normal(c["rows"], c["heads"] + 2 * c["kv_heads"], c["dim"], scale=3.0)
        s["q"], s["k"] = s["qkv"][:, :c["heads"]], s["qkv"][:, c["heads"]:c["heads"] + c["kv_heads"]]
        s["q_weight"], s["k_weight"] = (normal(c["dim"], scale=0.2).add_(1) for _ in range(2))
        s["positions"] = torch.randint(0, c["far"], (c["rows"],), generator=g, device=DEV, dtype=torch.int32)
        i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV)
        s["freq"] = torch.pow(1e6, -i / c["rot"]).float()
        s["eps"] = 1e-6
    elif c["op"] in ("window", "attend8"):
        ctx, n = _lengths(c["batch"], c["ctx_lo"], c["ctx_hi"]), _counts(c, "nodes")
        s["table"], pages = _table(rng, ctx, c["page"])
        shape = (pages, c["page"], c["kv_heads"], c["dim"])
        if c["op"] == "window":
            s["k"], s["v"] = normal(*shape), normal(*shape)
        else:
            (s["k"], s["k_scale"]), (s["v"], s["v_scale"]) = held8(*shape), held8(*shape)
        # queries twice a unit normal: logits of deviation 2, so that some keys take most of a row
        s["q"] = normal(sum(n), c["heads"], c["dim"], scale=2.0)
        s["k_new"] = normal(sum(n), c["kv_heads"], c["dim"])
        s["v_new"] = normal(sum(n), c["kv_heads"], c["dim"])
        s["cu"], s["ctx"], s["total"], s["longest"] = _cu(n), _i32(ctx), sum(n), max(ctx)
        s["mask"] = None if c["chain"] else _tree_masks(rng, n, -(-c["nodes"] // 32))
    else:
        ctx, n, acc = _lengths(c["batch"], c["ctx_lo"], c["ctx_hi"]), _counts(c, "nodes"), _accepted(c)
        s["table"], pages = _table(rng, [a + x for a, x in zip(ctx, n)], c["page"])
        shape = (c["layers"], pages, c["page"], c["kv_heads"], c["dim"])
        (s["k"], s["k_scale"]), (s["v"], s["v_scale"]) = held8(*shape), held8(*shape)
        s["k_new"] = normal(c["layers"], sum(n), c["kv_heads"], c["dim"])
        s["v_new"] = normal(c["layers"], sum(n), c["kv_heads"], c["dim"])
        path = np.full((c["batch"], c["nodes"]), -1, dtype=np.int32)
        for b, (x, a) in enumerate(zip(n, acc)):  # a path from the root: ascending nodes
            path[b, :a] = np.concatenate([[0], 1 + np.sort(rng.permutation(x - 1)[:a - 1])]) if x > 1 else [0]
        s["path"], s["path_len"] = torch.from_numpy(path).to(DEV), _i32(acc)
        s["cu"], s["ctx"], s["total"] = _cu(n), _i32(ctx), sum(n)
    if own:
        s["plan"] = _plan(s)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["op"]](state)


# the plain forms

def _norm(x, weight, eps):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()


def _rotate(s):
    angle = s["positions"].double()[:, None] * s["freq"].double()  # far positions leave 32 bits few of the turn's part
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot, out = s["rot"], {}
    for name in ("q", "k"):
        y = _norm(s[name], s[name + "_weight"], s["eps"])
        if s["pairs"] == "halves":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., :rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out[name] = torch.cat([turned, y[..., rot:]], -1).to(s["q"].dtype)
    return out


def _by_request(s, n):
    """Packed rows to [batch, n]: each place's row (a valid one everywhere), whether it is one, and the way back."""
    i = torch.arange(n, device=DEV)
    count = s["cu"][1:] - s["cu"][:-1]
    ok = i[None, :] < count[:, None]
    at = (s["cu"][:-1, None] + i[None, :]).clamp(max=s["total"] - 1).long()
    b = torch.repeat_interleave(torch.arange(s["batch"], device=DEV), count.long(), output_size=s["total"])
    return at, ok, (b, torch.arange(s["total"], device=DEV) - s["cu"][:-1].long()[b])


def _held(s, name, pos):
    """Cached keys or values at pos [batch, m], in 32 bits."""
    page, slot = torch.gather(s["table"], 1, pos // s["page"]).long(), pos % s["page"]
    if name + "_scale" not in s:
        return s[name][page, slot].float()
    x = s[name].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float()
    return x * s[name + "_scale"][page, slot // s["block"]][..., None]


def _attend(s):
    n, kv, window, sinks = s["nodes"], s["kv_heads"], s["window"], s["sinks"]
    at, ok, back = _by_request(s, n)
    ctx = s["ctx"][:, None].long()
    if window and window + sinks < s["longest"]:  # the first tokens and the last ones
        i = torch.arange(sinks + window, device=DEV)
        pos = torch.where(i < sinks, i, ctx - window + (i - sinks))
        real = (pos >= torch.where(i < sinks, 0, sinks)) & (pos < ctx)
    else:
        pos = torch.arange(s["longest"], device=DEV).expand(s["batch"], -1)
        real = pos < ctx
    pos = torch.where(real, pos, 0)
    k = torch.cat([_held(s, "k", pos), s["k_new"][at].float()], 1)
    q = s["q"][at].float().unflatten(2, (kv, -1))  # [b, n, kv, group, dim]
    z = torch.einsum("bnhgd,bahd->bhgna", q, k) * s["dim"] ** -0.5
    del k
    j = torch.arange(n, device=DEV)
    if s["mask"] is None:
        sees = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()[None].expand(s["batch"], n, n)
    else:
        sees = ((s["mask"][:, j // 32] >> (j % 32)) & 1).bool()[at]
    sees = sees & ok[:, None, :]
    old = real[:, None, :].expand(-1, n, -1)
    if window:
        place = ctx[:, :, None] + sees.cumsum(2) - 1  # each drafted token's place in the row's own text
        first = ctx[:, :, None] + sees.sum(2, keepdim=True) - window
        old = old & ((pos[:, None, :] < sinks) | (pos[:, None, :] >= first))
        sees = sees & ((place < sinks) | (place >= first))
    sees = torch.cat([old, sees], 2)[:, None, None]  # [b, 1, 1, n, keys + n]
    z = torch.where(sees, z, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (z - top).exp_()
    del z
    total = p.sum(-1, keepdim=True)
    v = torch.cat([_held(s, "v", pos), s["v_new"][at].float()], 1)
    o = torch.einsum("bhgna,bahd->bhgnd", p, v) / torch.where(total == 0, 1.0, total)
    out = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[back]
    lse = (total.log() + top)[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[back]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _power(top):
    """The smallest power of two whose 448-fold reaches `top` (0 for 0)."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), 0.0)


def _commit8(s):
    block, layers, heads = s["block"], s["layers"], s["kv_heads"]
    out = {"new_len": s["ctx"] + s["path_len"]}
    # places past a path's end repeat its last node: two places of one slot write the same
    i = torch.arange(s["nodes"], device=DEV).minimum(s["path_len"][:, None] - 1)
    node = (s["cu"][:-1, None] + torch.gather(s["path"], 1, i.long())).long()
    pos = (s["ctx"][:, None] + i).long()
    to = torch.gather(s["table"], 1, pos // s["page"]).long() * s["page"] + pos % s["page"]  # slots of the cache
    # the blocks that begin in earlier tokens: one a request at most
    begun = s["ctx"].long() % block
    first = to[:, 0] // block
    lane = torch.arange(block, device=DEV)
    for name in ("k", "v"):
        scale = s[name + "_scale"].flatten(1, 2)  # [layers, blocks, heads], a view
        held = s[name].view(torch.uint8).flatten(1, 2)  # [layers, slots, heads, dim], a view
        x = s[name + "_new"][:, node].float()  # [layers, batch, nodes, heads, dim]
        top = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
        where = (to // block)[None, :, :, None].expand(top.shape).flatten(1, 2)
        need = _power(torch.zeros_like(scale).scatter_reduce_(1, where, top.flatten(1, 2), "amax"))
        old = scale[:, first]
        new = scale.scatter(1, where, torch.gather(need, 1, where))
        grown = torch.where((begun > 0)[None, :, None], torch.maximum(old, need[:, first]), need[:, first])
        new[:, first] = grown
        # tokens that were there before, under the new scale
        slots = first[:, None] * block + lane
        was = held[:, slots].view(torch.float8_e4m3fn).float() * old[:, :, None, :, None]
        was = _to8(was, grown[:, :, None, :, None])
        mine = ((lane < begun[:, None])[None, :, :, None] & (grown > old)[:, :, None])[..., None]
        held[:, slots] = torch.where(mine, was, held[:, slots])
        held[:, to] = _to8(x, new[:, to // block][..., None])
        scale.copy_(new)
        out[name], out[name + "_scale"] = s[name], s[name + "_scale"]
    return out


def _to8(x, scale):
    """x / scale (a power of two where x is not zero) in e4m3, as bytes."""
    return (x * torch.where(scale > 0, 1 / scale, 0.0)).to(torch.float8_e4m3fn).view(torch.uint8)


_plain = {"rotate": _rotate, "window": _attend, "attend8": _attend, "commit8": _commit8}


# the package's calls

def _plan(s):
    """What a serving loop sets up once: the argument blocks, the workspace and the buffers of the results."""
    import speculative_decoding_verification_23_gb300 as sv

    def empty(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device=DEV)

    p = {"sv": sv}
    if s["op"] == "rotate":
        p["args"] = sv.make_rotate_args(q=s["q"], k=s["k"], positions=s["positions"], inv_freq=s["freq"],
                                        q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                                        interleaved=s["pairs"] == "neighbours")
        p["q"], p["k"] = (empty(*s[x].shape, dtype=s[x].dtype) for x in ("q", "k"))
        return p
    p["status"] = empty(s["batch"], dtype=torch.int32)
    if s["op"] == "window":
        p["args"] = sv.make_window_args(q=s["q"], k_new=s["k_new"], v_new=s["v_new"], cu_nodes=s["cu"],
                                        max_nodes=s["nodes"], tree_mask=s["mask"], cache=sv.make_cache(s["k"], s["v"]),
                                        block_table=s["table"], ctx_len=s["ctx"], window=s["window"], sinks=s["sinks"])
        p["workspace"] = sv.make_window_workspace(p["args"])
    else:
        cache = sv.make_cache8(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if s["op"] == "commit8":
            p["args"] = sv.make_cache8_commit_args(k_new=s["k_new"], v_new=s["v_new"], cu_nodes=s["cu"], path=s["path"],
                                                   path_len=s["path_len"], cache=cache, block_table=s["table"],
                                                   ctx_len=s["ctx"])
            p["new_len"] = empty(s["batch"], dtype=torch.int32)
            return p
        p["args"] = sv.make_cache8_args(q=s["q"], k_new=s["k_new"], v_new=s["v_new"], cu_nodes=s["cu"],
                                        max_nodes=s["nodes"], tree_mask=s["mask"], cache=cache, block_table=s["table"],
                                        ctx_len=s["ctx"], window=s["window"], sinks=s["sinks"])
        p["workspace"] = sv.make_cache8_workspace(p["args"])
    p["out"], p["lse"] = torch.empty_like(s["q"]), empty(s["total"], s["heads"], dtype=torch.float32)
    return p


def _own_rotate(s):
    p = s["plan"]
    q, k = p["sv"].spec_norm_rotate(p["args"], out_q=p["q"], out_k=p["k"])
    return {"q": q, "k": k}


def _own_window(s):
    p = s["plan"]
    out, lse, _ = p["sv"].spec_window_attention(p["args"], workspace=p["workspace"], out=p["out"], out_lse=p["lse"],
                                                out_status=p["status"])
    return {"out": out, "lse": lse}


def _own_attend8(s):
    p = s["plan"]
    out, lse, _ = p["sv"].spec_cache8_attention(p["args"], workspace=p["workspace"], out=p["out"], out_lse=p["lse"],
                                                out_status=p["status"])
    return {"out": out, "lse": lse}


def _own_commit8(s):
    p = s["plan"]
    new_len, _ = p["sv"].spec_cache8_commit(p["args"], out_len=p["new_len"], out_status=p["status"])
    return {"new_len": new_len, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


_own = {"rotate": _own_rotate, "window": _own_window, "attend8": _own_attend8, "commit8": _own_commit8}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return _exact[case["op"]](s)


def _exact_rotate(s):
    turns = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                        torch.outer(s["positions"].double(), s["freq"].double()))[:, None]  # e^(i angle)
    rot, half = s["rot"], s["rot"] // 2
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = s[name + "_weight"].double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / s["dim"] + s["eps"])
        place = torch.arange(rot, device=DEV)
        place = (place.view(2, half).T if s["pairs"] == "halves" else place.view(half, 2)).contiguous()
        z = torch.view_as_complex(y[..., place].contiguous()) * turns
        y[..., place] = torch.view_as_real(z)
        out[name] = y
    return out


def _keys(s, name, b, length):
    pos = torch.arange(length, device=DEV)
    page, slot = s["table"][b, pos // s["page"]].long(), pos % s["page"]
    if s["op"] == "window":
        return s[name][page, slot].double()
    x = s[name].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).double()
    return x * s[name + "_scale"][page, slot // s["block"]].double()[..., None]


def _exact_attend(s):
    outs, lses = [], []
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    group = s["heads"] // s["kv_heads"]
    for b in range(s["batch"]):
        lo, hi = cu[b], cu[b + 1]
        n, a = hi - lo, ctx[b]
        k = torch.cat([_keys(s, "k", b, a), s["k_new"][lo:hi].double()])
        v = torch.cat([_keys(s, "v", b, a), s["v_new"][lo:hi].double()])
        rows = np.zeros((n, a + n), dtype=bool)
        masks = None if s["mask"] is None else s["mask"][lo:hi].cpu().numpy().astype(np.int64) & 0xFFFFFFFF
        for i in range(n):
            seen = [j for j in range(n) if (j <= i if masks is None else masks[i, j // 32] >> (j % 32) & 1)]
            text = np.concatenate([np.arange(a), a + np.array(seen, dtype=np.int64)])  # all that it would see, in order
            if s["window"] and s["window"] + s["sinks"] < len(text):
                text = np.concatenate([text[:s["sinks"]], text[-s["window"]:]])
            rows[i, text] = True
        sees = torch.from_numpy(rows).to(DEV)
        some = sees.any(0)
        k, v, sees = k[some], v[some], sees[:, some]
        o = torch.zeros(n, s["heads"], s["dim"], dtype=torch.float64, device=DEV)
        e = torch.zeros(n, s["heads"], dtype=torch.float64, device=DEV)
        for h in range(s["heads"]):
            z = s["q"][lo:hi, h].double() @ k[:, h // group].T / math.sqrt(s["dim"])
            z[~sees] = -math.inf
            e[:, h] = torch.logsumexp(z, 1)
            o[:, h] = torch.exp(z - e[:, h, None]) @ v[:, h // group]
        outs.append(o)
        lses.append(e)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _nearest8(x):
    """The e4m3 value nearest to each of x, ties to the even one: steps of 2^(e-3), at least 2^-9."""
    e = torch.floor(torch.log2(torch.clamp(x.abs(), min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_commit8(s):
    cu, ctx, page, block = s["cu"].tolist(), s["ctx"].tolist(), s["page"], s["block"]
    table, path = s["table"].cpu().numpy(), s["path"].cpu().numpy()
    out, new = {}, []
    for name in ("k", "v"):
        held, scale = s[name].double(), s[name + "_scale"].double()
        for b, m in enumerate(s["path_len"].tolist()):
            x = s[name + "_new"][:, torch.from_numpy((cu[b] + path[b, :m]).astype(np.int64)).to(DEV)].double()
            at = ctx[b]
            while at < ctx[b] + m:  # a block at a time
                p, j = int(table[b, at // page]), at % page // block
                end = min(ctx[b] + m, at - at % block + block)
                part = x[:, at - ctx[b]:end - ctx[b]]  # [layers, tokens, heads, dim]
                top = part.abs().amax((1, 3))
                want = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
                was = scale[:, p, j].clone()
                if at % block:
                    want = torch.maximum(want, was)
                    lo = at % page - at % block
                    old = held[:, p, lo:at % page]
                    again = _nearest8(old * (was / want)[:, None, :, None])
                    held[:, p, lo:at % page] = torch.where((want > was)[:, None, :, None], again, old)
                scale[:, p, j] = want
                held[:, p, at % page:at % page + end - at] = _nearest8(part / want[:, None, :, None])
                at = end
            if name == "k":
                new.append(ctx[b] + m)
        out[name], out[name + "_scale"] = held, scale
    return {**out, "new_len": np.array(new, dtype=np.int32)}


_exact = {"rotate": _exact_rotate, "window": _exact_attend, "attend8": _exact_attend, "commit8": _exact_commit8}
