"""Measured cases of the drafted-tree operators: attention of a drafted tree over a paged cache, accumulation of
attention weights, eviction from the cache, commitment of the accepted path, and beam selection with reordering.

Each case is one call (for the beams: a selection and the reordering that follows it) as a serving loop makes it, on
the inputs that such a loop has in hand.  `own` false computes the plain form, elementary torch operations in 32 bits
(64 where an order hangs on the last bits); `own` true makes the package's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of a small draft model (14 heads in 2 groups of 64), one request: the drafter's own step
        dict(name="attend one token", op="attend", batch=1, nodes=1, ragged=False, chain=True, heads=14, kv_heads=2,
             dim=64, ctx_lo=1001, ctx_hi=1001, page=16, dtype="bf16"),
        # K = 8 drafts and the last token for 64 ragged requests, 28 heads in 4 groups of 128: the verify step
        dict(name="attend chains", op="attend", batch=64, nodes=9, ragged=True, chain=True, heads=28, kv_heads=4,
             dim=128, ctx_lo=257, ctx_hi=4096, page=16, dtype="bf16"),
        # trees of up to 64 drafted tokens, a middle batch of long chats, half precision, large pages
        dict(name="attend trees", op="attend", batch=16, nodes=64, ragged=True, chain=False, heads=32, kv_heads=8,
             dim=128, ctx_lo=1024, ctx_hi=8191, page=64, dtype="fp16"),
        # two documents of up to 128 K tokens with a tree of 32: the longest contexts
        dict(name="attend long", op="attend", batch=2, nodes=32, ragged=False, chain=False, heads=16, kv_heads=8,
             dim=128, ctx_lo=100003, ctx_hi=131072, page=32, dtype="bf16"),
        # the weights that one request's accepted tokens put on its cache
        dict(name="weigh one request", op="weigh", batch=1, rows=5, ragged=False, heads=28, kv_heads=4, dim=128,
             len_lo=4001, len_hi=4001, page=16, dtype="bf16"),
        # the same for a batch of long requests
        dict(name="weigh a batch", op="weigh", batch=16, rows=9, ragged=True, heads=32, kv_heads=8, dim=128,
             len_lo=2048, len_hi=16384, page=64, dtype="bf16"),
        # one request's cache cut from 4000 tokens to 1024
        dict(name="evict one request", op="evict", batch=1, kv_heads=2, dim=64, len_lo=4001, len_hi=4001, keep=1024,
             sink=4, recent=128, page=16, dtype="bf16"),
        # a batch cut to 2000 tokens a head
        dict(name="evict a batch", op="evict", batch=16, kv_heads=8, dim=128, len_lo=1500, len_hi=16384, keep=2000,
             sink=4, recent=256, page=64, dtype="fp16"),
        # one request's accepted path written to every layer of the draft model's cache
        dict(name="commit one request", op="commit", layers=24, batch=1, nodes=9, ragged=False, kv_heads=2, dim=64,
             ctx_lo=777, ctx_hi=777, page=16, dtype="bf16"),
        # 64 requests' paths, all 28 layers of the target's cache
        dict(name="commit a batch", op="commit", layers=28, batch=64, nodes=33, ragged=True, kv_heads=4, dim=128,
             ctx_lo=100, ctx_hi=1000, page=16, dtype="bf16"),
        # one request's tree grown by a level: 4 nodes of 151936 logits to 4 children
        dict(name="beams of one request", op="beams", batch=1, beams=4, keep=4, vocab=151936, finished=False,
             history=64, state=896, dtype="bf16"),
        # 64 requests of 8 beams, the whole vocabulary, some beams ended
        dict(name="beams of a batch", op="beams", batch=64, beams=8, keep=8, vocab=152064, finished=True,
             history=500, state=3584, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "weigh", "evict", "commit", "beams", "beams"])
    limit = [work(c) for c in listed() if c["op"] == op]
    most = {k: max(w[k] for w in limit) for k in ("bytes", "flops")}
    while True:
        kv = rng.choice([1, 2, 4, 8])
        c = dict(op=op, batch=_log(rng, 1, 64))
        if op in ("attend", "weigh"):
            hi = _log(rng, 64, 131072)
            c.update(nodes=_log(rng, 1, 64)) if op == "attend" else c.update(rows=_log(rng, 1, 32))
            c.update(ragged=rng.random() < 0.5, heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8]), kv_heads=kv)
            c.update(dim=rng.choice([64, 128]))
            if op == "attend":
                c.update(chain=rng.random() < 0.4, ctx_lo=rng.choice([0, hi // 8, hi]), ctx_hi=hi)
            else:
                c.update(len_lo=max(c["rows"], rng.choice([hi // 8, hi])), len_hi=max(c["rows"], hi))
        elif op == "evict":
            hi = _log(rng, 200, 65536)
            keep = _log(rng, 64, max(64, hi // 2))
            c.update(kv_heads=kv, dim=rng.choice([64, 128]), len_lo=rng.choice([hi // 8, hi]), len_hi=hi, keep=keep)
            c.update(sink=rng.choice([0, 4]), recent=rng.randrange(0, keep // 2 + 1))
        elif op == "commit":
            hi = _log(rng, 16, 4096)
            c.update(layers=_log(rng, 1, 32), nodes=_log(rng, 1, 64), ragged=rng.random() < 0.5, kv_heads=kv)
            c.update(dim=rng.choice([64, 128]), ctx_lo=hi // 2, ctx_hi=hi)
        else:
            c.update(beams=_log(rng, 1, 32), keep=_log(rng, 1, 32), vocab=_log(rng, 500, 152064))
            c.update(finished=rng.random() < 0.5, history=_log(rng, 8, 2048), state=8 * _log(rng, 8, 512))
            c["keep"] = min(c["keep"], c["vocab"] // 2)
        if op != "beams":
            c["page"] = rng.choice([16, 32, 64, 128])
            c["dtype"] = rng.choice(["bf16", "fp16"])
        else:
            c["dtype"] = rng.choice(["bf16", "fp32"])
        w = work(c)
        if all(w[k] <= most[k] for k in most) and _plain_bytes(c) <= 8 << 30:
            return c


def _plain_bytes(c):
    """What the plain form holds at once, roughly: its padded copies in 32 bits."""
    if c["op"] == "attend":
        return c["batch"] * (c["ctx_hi"] + c["nodes"]) * 4 * (2 * c["kv_heads"] * c["dim"] + 2 * c["heads"] * c["nodes"])
    if c["op"] == "weigh":
        return c["batch"] * c["len_hi"] * 4 * (c["kv_heads"] * c["dim"] + 2 * c["heads"] * c["rows"])
    if c["op"] == "evict":
        return c["batch"] * c["kv_heads"] * (c["len_hi"] * 16 + c["keep"] * c["dim"] * 8)
    return 0


def _lengths(n, lo, hi):
    """n whole numbers of lo..hi, ragged and always the same ones; the last is hi."""
    return [lo + ((i * 2654435761 + 1013904223) % (1 << 32)) * (hi - lo + 1) // (1 << 32) for i in range(n - 1)] + [hi]


def _counts(c, key):
    return _lengths(c["batch"], max(1, c[key] // 2) if c["ragged"] else c[key], c[key])


def work(c):
    es = BYTES[c["dtype"]]
    if c["op"] == "attend":
        ctx, n = _lengths(c["batch"], c["ctx_lo"], c["ctx_hi"]), _counts(c, "nodes")
        pairs = sum(a * b for a, b in zip(ctx, n)) + sum(n)  # a drafted token sees itself at least
        kv = (sum(ctx) + sum(n)) * c["kv_heads"] * c["dim"] * 2 * es
        return {"bytes": kv + sum(n) * c["heads"] * (2 * c["dim"] * es + 4), "flops": 4 * c["dim"] * c["heads"] * pairs}
    if c["op"] == "weigh":
        ln, n = _lengths(c["batch"], c["len_lo"], c["len_hi"]), _counts(c, "rows")
        pairs = sum(r * (a - r) + r * (r + 1) // 2 for a, r in zip(ln, n))
        keys = sum(ln) * c["kv_heads"] * (c["dim"] * es + 4 + 4)
        return {"bytes": keys + sum(n) * c["heads"] * (c["dim"] * es + 4), "flops": 2 * c["dim"] * c["heads"] * pairs}
    if c["op"] == "evict":
        ln = _lengths(c["batch"], c["len_lo"], c["len_hi"])
        kept = sum(min(a, c["keep"]) for a in ln)
        return {"bytes": c["kv_heads"] * (sum(ln) * 4 + kept * (4 * c["dim"] * es + 8)), "flops": c["kv_heads"] * sum(ln)}
    if c["op"] == "commit":
        kept = sum(max(1, n // 2) for n in _counts(c, "nodes"))
        return {"bytes": c["layers"] * kept * c["kv_heads"] * c["dim"] * 4 * es, "flops": 0}
    rows = c["batch"] * c["beams"]
    moved = c["batch"] * c["keep"] * 2 * (c["history"] * 4 + c["state"] * 2)
    return {"bytes": rows * c["vocab"] * es + rows * 4 + c["batch"] * c["keep"] * 12 + moved, "flops": 3 * rows * c["vocab"]}


# ------------------------------------------------------------------ the inputs

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cu(counts):
    return _i32(np.concatenate([[0], np.cumsum(counts)]).tolist())


def _table(rng, lens, page, first=0):
    """A block table of scattered pages for these lengths, and the number of pages."""
    need = [-(-n // page) for n in lens]
    ids = first + rng.permutation(sum(need))
    width, at = max(1, max(need)), 0
    table = np.zeros((len(lens), width), dtype=np.int32)
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(table).to(DEV), sum(need)


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

    s = dict(c)
    if c["op"] == "attend":
        ctx, n = _lengths(c["batch"], c["ctx_lo"], c["ctx_hi"]), _counts(c, "nodes")
        s["table"], pages = _table(rng, ctx, c["page"])
        s["k"] = normal(max(1, pages), c["page"], c["kv_heads"], c["dim"])
        s["v"] = normal(max(1, pages), c["page"], c["kv_heads"], c["dim"])
        # queries twice a unit normal: logits of deviation 2, so that some keys take most of a row
        s["q"] = normal(sum(n), c["heads"], c["dim"], scale=2.0)
        s["k_new"] = normal(sum(n), c["kv_heads"], c["dim"])
        s["v_new"] = normal(sum(n), c["kv_heads"], c["dim"])
        s["cu"], s["ctx"], s["total"], s["longest"] = _cu(n), _i32(ctx), sum(n), max(ctx)
        s["mask"] = None if c["chain"] else _tree_masks(rng, n, -(-c["nodes"] // 32))
    elif c["op"] == "weigh":
        ln, n = _lengths(c["batch"], c["len_lo"], c["len_hi"]), _counts(c, "rows")
        s["table"], pages = _table(rng, ln, c["page"])
        s["k"] = normal(pages, c["page"], c["kv_heads"], c["dim"])
        s["v"] = s["k"]  # the values are not read
        s["q"] = normal(sum(n), c["heads"], c["dim"], scale=2.0)
        s["cu"], s["len"], s["total"], s["longest"] = _cu(n), _i32(ln), sum(n), max(ln)
        # the weights of the rounds before, and what the attention of this round gave beside its output
        s["before"] = normal(c["batch"], c["kv_heads"], max(ln), dtype=torch.float32).exp_()
        s["lse"] = _row_lse(s)
    elif c["op"] == "evict":
        ln = _lengths(c["batch"], c["len_lo"], c["len_hi"])
        s["table"], pages = _table(rng, ln, c["page"])
        s["to_table"], more = _table(rng, [min(a, c["keep"]) for a in ln], c["page"], pages)
        s["first"] = pages
        s["k"] = normal(pages + more, c["page"], c["kv_heads"], c["dim"])
        s["v"] = normal(pages + more, c["page"], c["kv_heads"], c["dim"])
        # accumulated weights have a long tail; one in ten is still at zero
        w = normal(c["batch"], c["kv_heads"], max(ln), dtype=torch.float32, scale=2.0).exp_()
        s["weights"] = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.1, torch.zeros_like(w), w)
        s["len"] = _i32(ln)
    elif c["op"] == "commit":
        ctx, n = _lengths(c["batch"], c["ctx_lo"], c["ctx_hi"]), _counts(c, "nodes")
        acc = [max(1, x // 2) for x in n]
        s["table"], pages = _table(rng, [a + x for a, x in zip(ctx, n)], c["page"])
        s["k"] = normal(c["layers"], pages, c["page"], c["kv_heads"], c["dim"])
        s["v"] = normal(c["layers"], pages, c["page"], c["kv_heads"], c["dim"])
        s["k_new"] = normal(c["layers"], sum(n), c["kv_heads"], c["dim"])
        s["v_new"] = normal(c["layers"], sum(n), c["kv_heads"], c["dim"])
        path = np.full((c["batch"], c["nodes"]), -1, dtype=np.int32)
        for b, (x, a) in enumerate(zip(n, acc)):  # a path from the root: ascending nodes
            path[b, :a] = np.concatenate([[0], 1 + np.sort(rng.permutation(x - 1)[:a - 1])]) if x > 1 else [0]
        s["path"], s["path_len"] = torch.from_numpy(path).to(DEV), _i32(acc)
        s["cu"], s["ctx"], s["total"] = _cu(n), _i32(ctx), sum(n)
    else:
        b, w, v = c["batch"], c["beams"], c["vocab"]
        # a vocabulary's bias that falls with the token's rank, and a row's own part
        bias = -1.1 * torch.log(torch.arange(1, v + 1, device=DEV, dtype=torch.float32))
        bias = bias[torch.randperm(v, generator=g, device=DEV)]
        s["logits"] = torch.empty(b * w, v + (-v) % 8, dtype=t, device=DEV)
        s["logits"].normal_(generator=g).mul_(3.0)[:, :v].add_(bias.to(t))
        s["scores"] = -5.0 * torch.rand(b, w, generator=g, device=DEV)
        s["ended"] = (torch.rand(b, w, generator=g, device=DEV) < 0.2).to(torch.int32) if c["finished"] else None
        s["ids"] = torch.randint(0, v, (b, w, c["history"]), generator=g, device=DEV, dtype=torch.int32)
        s["hidden"] = normal(b, w, c["state"], dtype=torch.bfloat16)
        s["ids_out"] = torch.empty(b, c["keep"], c["history"], dtype=torch.int32, device=DEV)
        s["hidden_out"] = torch.empty(b, c["keep"], c["state"], dtype=torch.bfloat16, device=DEV)
    if own:
        s["plan"] = _plan(s)
    return s


def _row_lse(s):
    """Each row's log of its softmax's sum, as the attention returns it ([total, heads], 32 bits)."""
    lse, scale = [], s["dim"] ** -0.5
    cu, ln = s["cu"].tolist(), s["len"].tolist()
    for b in range(s["batch"]):
        n, a = cu[b + 1] - cu[b], ln[b]
        k = s["k"][s["table"][b].long()].flatten(0, 1)[:a].float()  # [a, kv_heads, dim]
        q = s["q"][cu[b]:cu[b + 1]].float().unflatten(1, (s["kv_heads"], -1))
        z = torch.einsum("nhgd,ahd->nhga", q, k) * scale
        late = torch.arange(a, device=DEV)[None, :] > torch.arange(a - n, a, device=DEV)[:, None]
        lse.append(z.masked_fill_(late[:, None, None, :], -math.inf).logsumexp(-1).flatten(1))
    return torch.cat(lse).contiguous()


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["op"]](state)


# the plain forms

def _by_request(s, n):
    """Packed rows to [batch, n]: each place's row (a valid one everywhere), whether it is one, and the way back."""
    i = torch.arange(n, device=DEV)
    count = s["cu"][1:] - s["cu"][:-1]
    ok = i[None, :] < count[:, None]
    at = (s["cu"][:-1, None] + i[None, :]).clamp(max=s["total"] - 1).long()
    b = torch.repeat_interleave(torch.arange(s["batch"], device=DEV), count.long(), output_size=s["total"])
    return at, ok, (b, torch.arange(s["total"], device=DEV) - s["cu"][:-1].long()[b]), count


def _attend(s):
    n, kv, a = s["nodes"], s["kv_heads"], s["longest"]
    at, ok, back, _ = _by_request(s, n)
    q = s["q"][at].float().unflatten(2, (kv, -1))  # [b, n, kv, group, dim]
    k = torch.cat([s["k"][s["table"].long()].flatten(1, 2)[:, :a], s["k_new"][at]], 1).float()
    z = torch.einsum("bnhgd,bahd->bhgna", q, k) * s["dim"] ** -0.5
    del k
    if s["mask"] is None:
        sees = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()[None].expand(s["batch"], n, n)
    else:
        j = torch.arange(n, device=DEV)
        sees = ((s["mask"][:, j // 32] >> (j % 32)) & 1).bool()[at]
    old = (torch.arange(a, device=DEV)[None, :] < s["ctx"][:, None])[:, None, :].expand(s["batch"], n, a)
    sees = torch.cat([old, sees & ok[:, None, :]], 2)[:, None, None]  # [b, 1, 1, n, a + n]
    z = torch.where(sees, z, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (z - top).exp_()
    del z
    total = p.sum(-1, keepdim=True)
    v = torch.cat([s["v"][s["table"].long()].flatten(1, 2)[:, :a], s["v_new"][at]], 1)
    v = torch.where((torch.cat([old[:, 0], ok], 1))[:, :, None, None], v, torch.zeros_like(v)).float()
    o = torch.einsum("bhgna,bahd->bhgnd", p, v) / torch.where(total == 0, 1.0, total)
    out = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[back]
    lse = (total.log() + top)[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[back]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _weigh(s):
    n, kv, a = s["rows"], s["kv_heads"], s["longest"]
    at, ok, _, count = _by_request(s, n)
    q = s["q"][at].float().unflatten(2, (kv, -1))
    k = s["k"][s["table"].long()].flatten(1, 2)[:, :a].float()
    z = torch.einsum("bnhgd,bahd->bhgna", q, k) * s["dim"] ** -0.5
    lse = s["lse"][at].unflatten(2, (kv, -1)).permute(0, 2, 3, 1)[..., None]
    j, i = torch.arange(a, device=DEV), torch.arange(n, device=DEV)
    sees = (j[None, None, :] <= (s["len"] - count)[:, None, None] + i[None, :, None]) & ok[:, :, None]
    p = torch.where(sees[:, None, None], (z - lse).exp_(), 0.0)
    w = s["before"] + p.sum((2, 3))
    return {"weights": torch.where((j[None, :] < s["len"][:, None])[:, None], w, 0.0)}


def _put(cache, table, page, pos, values, heads):
    """cache[page of pos, slot of pos, head] = values.  Places that repeat a position repeat its values."""
    at = torch.gather(table, 1, (pos.flatten(1) // page).long()).view(pos.shape) * page + pos % page
    cache.view(-1, *cache.shape[2:])[at.long(), heads] = values


def _evict(s):
    w, keep, page = s["weights"], s["keep"], s["page"]
    j = torch.arange(w.shape[2], device=DEV)
    ln = s["len"][:, None, None]
    safe = (j < s["sink"]) | (j >= ln - s["recent"])
    key = torch.where(j < ln, torch.where(safe, math.inf, w), -math.inf)
    by = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :keep]
    if by.shape[2] < keep:
        by = torch.cat([by, by.new_full((*by.shape[:2], keep - by.shape[2]), 1 << 30)], 2)
    new_len = s["len"].clamp(max=keep)
    i = torch.arange(keep, device=DEV)
    ok = (i < new_len[:, None, None]).expand(by.shape)
    index = torch.sort(torch.where(ok, by, 1 << 30), dim=2).values
    index = torch.where(ok, index, -1)
    src = index.clamp(min=0)
    kept = torch.where(ok, torch.gather(w, 2, src), 0.0)
    # what is moved: places past the kept tokens repeat the last of them
    to = i.minimum(new_len[:, None, None] - 1).expand(by.shape)
    src = torch.gather(src, 2, to.long())
    heads = torch.arange(s["kv_heads"], device=DEV)[None, :, None].expand(by.shape)
    at = torch.gather(s["table"], 1, (src // page).flatten(1)).view(src.shape) * page + src % page
    for name in ("k", "v"):
        values = s[name].view(-1, *s[name].shape[2:])[at.long(), heads]
        _put(s[name], s["to_table"], page, to, values, heads)
    return {"index": index.int(), "kept": kept, "new_len": new_len, "k": s["k"][s["first"]:], "v": s["v"][s["first"]:]}


def _commit(s):
    # places past a path's end repeat its last node: two places of one slot write the same
    i = torch.arange(s["nodes"], device=DEV).minimum(s["path_len"][:, None] - 1)
    at = (s["cu"][:-1, None] + torch.gather(s["path"], 1, i.long())).long()
    pos = s["ctx"][:, None] + i
    to = (torch.gather(s["table"], 1, (pos // s["page"]).long()) * s["page"] + pos % s["page"]).long()
    for name in ("k", "v"):
        s[name].flatten(1, 2)[:, to] = s[name + "_new"][:, at]  # a view: layers, slots, heads, dim
    return {"k": s["k"], "v": s["v"], "new_len": s["ctx"] + s["path_len"]}


def _beams(s):
    b, w, v, keep = s["batch"], s["beams"], s["vocab"], s["keep"]
    z = s["logits"][:, :v].double()  # the order of two beams' scores can hang on the last bits of 32
    z -= z.amax(1, keepdim=True)
    z -= z.exp().sum(1, keepdim=True).log_()
    total = (s["scores"].double()[:, :, None] + z.view(b, w, v))
    if s["ended"] is not None:  # an ended beam goes on as it is, through its end token (0)
        first = torch.arange(v, device=DEV) == 0
        ended = s["ended"].bool()[:, :, None]
        total = torch.where(ended, torch.where(first, s["scores"].double()[:, :, None], -math.inf), total)
    flat = total.view(b, w * v)
    # all candidates from the last kept score on, in their own order, then sorted with ties to the lowest
    room = keep + 512
    last = torch.topk(flat, keep, dim=1).values[:, -1:]
    place = torch.cumsum(flat >= last, 1)
    place = torch.where((flat >= last) & (place <= room), place, 0)
    some = torch.full((b, room + 1), w * v, dtype=torch.int64, device=DEV)
    some.scatter_(1, place, torch.arange(w * v, device=DEV).expand(b, w * v))
    some = some[:, 1:]
    val = torch.where(some < w * v, torch.gather(flat, 1, some.clamp(max=w * v - 1)), -math.inf)
    val, by = torch.sort(val, dim=1, descending=True, stable=True)
    pick = torch.gather(some, 1, by[:, :keep])
    parent, token = pick // v, pick % v
    rows = torch.arange(b, device=DEV)[:, None]
    return {"scores": val[:, :keep].float(), "parents": parent.int(), "tokens": token.int(),
            "ids": s["ids"][rows, parent], "hidden": s["hidden"][rows, parent]}


_plain = {"attend": _attend, "weigh": _weigh, "evict": _evict, "commit": _commit, "beams": _beams}


# the package's calls

def _plan(s):
    """What a serving loop sets up once: the argument blocks, the workspace and the buffers of the results."""
    import speculative_decoding_verification_23_gb300 as sv

    def empty(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device=DEV)

    b = s["batch"]
    p = {"sv": sv, "status": empty(b, dtype=torch.int32)}
    if s["op"] == "beams":
        p["args"] = sv.make_beam_args(logits=s["logits"], V=s["vocab"], scores=s["scores"], keep=s["keep"],
                                      finished=s["ended"], end_token=0)
        p["parents"], p["tokens"] = (empty(b, s["keep"], dtype=torch.int32) for _ in range(2))
        p["scores"] = empty(b, s["keep"], dtype=torch.float32)
        p["move"] = sv.make_reorder_args(parents=p["parents"], beams=s["beams"],
                                         states=[(s["ids"], s["ids_out"]), (s["hidden"], s["hidden_out"])])
        p["workspace"] = sv.make_beam_workspace(p["args"])
        return p
    p["cache"] = cache = sv.make_cache(s["k"], s["v"])
    if s["op"] == "attend":
        p["args"] = sv.make_tree_args(q=s["q"], k_new=s["k_new"], v_new=s["v_new"], cu_nodes=s["cu"],
                                      max_nodes=s["nodes"], tree_mask=s["mask"], cache=cache, block_table=s["table"],
                                      ctx_len=s["ctx"])
        p["workspace"] = sv.make_tree_workspace(p["args"])
        p["out"], p["lse"] = torch.empty_like(s["q"]), empty(s["total"], s["heads"], dtype=torch.float32)
    elif s["op"] == "weigh":
        p["args"] = sv.make_weigh_args(q=s["q"], lse=s["lse"], cu_rows=s["cu"], max_rows=s["rows"], cache=cache,
                                       block_table=s["table"], kv_len=s["len"])
        p["weights"] = torch.empty_like(s["before"])
    elif s["op"] == "evict":
        p["args"] = sv.make_evict_args(weights=s["weights"], kv_len=s["len"], keep=s["keep"], sink=s["sink"],
                                       recent=s["recent"], cache=cache, block_table=s["table"],
                                       to_table=s["to_table"])
        p["index"] = empty(b, s["kv_heads"], s["keep"], dtype=torch.int32)
        p["kept"] = empty(b, s["kv_heads"], s["keep"], dtype=torch.float32)
        p["new_len"] = empty(b, dtype=torch.int32)
    else:
        p["args"] = sv.make_commit_args(k_new=s["k_new"], v_new=s["v_new"], cu_nodes=s["cu"], path=s["path"],
                                        path_len=s["path_len"], cache=cache, block_table=s["table"], ctx_len=s["ctx"])
        p["new_len"] = empty(b, dtype=torch.int32)
    return p


def _own_attend(s):
    p = s["plan"]
    out, lse, _ = p["sv"].spec_tree_attention(p["args"], workspace=p["workspace"], out=p["out"], out_lse=p["lse"],
                                              out_status=p["status"])
    return {"out": out, "lse": lse}


def _own_weigh(s):
    p = s["plan"]
    w, _ = p["sv"].spec_attention_weights(p["args"], s["before"], out=p["weights"], out_status=p["status"])
    return {"weights": w}


def _own_evict(s):
    p = s["plan"]
    index, kept, new_len, _ = p["sv"].spec_cache_evict(p["args"], out_index=p["index"], out_kept=p["kept"],
                                                       out_len=p["new_len"], out_status=p["status"])
    return {"index": index, "kept": kept, "new_len": new_len, "k": s["k"][s["first"]:], "v": s["v"][s["first"]:]}


def _own_commit(s):
    p = s["plan"]
    new_len, _ = p["sv"].spec_cache_commit(p["args"], out_len=p["new_len"], out_status=p["status"])
    return {"k": s["k"], "v": s["v"], "new_len": new_len}


def _own_beams(s):
    p = s["plan"]
    scores, parents, tokens, _ = p["sv"].spec_beam_select(
        p["args"], workspace=p["workspace"], out_scores=p["scores"], out_parents=p["parents"], out_tokens=p["tokens"],
        out_status=p["status"])
    p["sv"].spec_beam_reorder(p["move"])
    return {"scores": scores, "parents": parents, "tokens": tokens, "ids": s["ids_out"], "hidden": s["hidden_out"]}


_own = {"attend": _own_attend, "weigh": _own_weigh, "evict": _own_evict, "commit": _own_commit, "beams": _own_beams}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return _exact[case["op"]](s)


def _keys(s, name, b, length):
    pos = torch.arange(length, device=DEV)
    return s[name][s["table"][b, pos // s["page"]].long(), pos % s["page"]].double()


def _exact_attend(s):
    outs, lses = [], []
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    group = s["heads"] // s["kv_heads"]
    for b in range(s["batch"]):
        lo, hi = cu[b], cu[b + 1]
        n = hi - lo
        k = torch.cat([_keys(s, "k", b, ctx[b]), s["k_new"][lo:hi].double()])
        v = torch.cat([_keys(s, "v", b, ctx[b]), s["v_new"][lo:hi].double()])
        sees = torch.zeros(n, ctx[b] + n, dtype=torch.bool, device=DEV)
        sees[:, :ctx[b]] = True
        for i in range(n):
            bits = (1 << (i + 1)) - 1
            if s["mask"] is not None:
                bits = sum((int(x) & 0xFFFFFFFF) << (32 * w) for w, x in enumerate(s["mask"][lo + i].tolist()))
            sees[i, ctx[b]:] = torch.tensor([bool(bits >> j & 1) for j in range(n)], device=DEV)
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


def _exact_weigh(s):
    w = torch.zeros(s["before"].shape, dtype=torch.float64, device=DEV)
    cu, ln = s["cu"].tolist(), s["len"].tolist()
    group = s["heads"] // s["kv_heads"]
    for b in range(s["batch"]):
        n, a = cu[b + 1] - cu[b], ln[b]
        k = _keys(s, "k", b, a)
        w[b, :, :a] = s["before"][b, :, :a].double()
        for h in range(s["heads"]):
            z = s["q"][cu[b]:cu[b + 1], h].double() @ k[:, h // group].T / math.sqrt(s["dim"])
            p = torch.exp(z - s["lse"][cu[b]:cu[b + 1], h, None].double())
            for i in range(n):
                p[i, a - n + i + 1:] = 0
            w[b, h // group, :a] += p.sum(0)
    return {"weights": w}


def _exact_evict(s):
    b, h, keep = s["batch"], s["kv_heads"], s["keep"]
    index = np.full((b, h, keep), -1, dtype=np.int32)
    kept = np.zeros((b, h, keep))
    k, v = s["k"].double(), s["v"].double()
    weights, table, to = s["weights"].cpu().numpy(), s["table"].cpu().numpy(), s["to_table"].cpu().numpy()
    lens = s["len"].tolist()
    for i, a in enumerate(lens):
        m = min(a, keep)
        for g in range(h):
            key = weights[i, g, :a].astype(np.float64)
            key[:s["sink"]] = np.inf
            key[max(0, a - s["recent"]):] = np.inf
            best = np.sort(np.lexsort((np.arange(a), -key))[:m])
            index[i, g, :m], kept[i, g, :m] = best, weights[i, g, best]
            new = np.arange(m)
            src = [torch.from_numpy(x.astype(np.int64)).to(DEV) for x in (table[i, best // s["page"]], best % s["page"])]
            dst = [torch.from_numpy(x.astype(np.int64)).to(DEV) for x in (to[i, new // s["page"]], new % s["page"])]
            for c in (k, v):
                c[dst[0], dst[1], g] = c[src[0], src[1], g]
    return {"index": index, "kept": kept, "new_len": np.minimum(lens, keep).astype(np.int32),
            "k": k[s["first"]:], "v": v[s["first"]:]}


def _exact_commit(s):
    k, v = s["k"].double(), s["v"].double()
    cu, ctx, table, path = s["cu"].tolist(), s["ctx"].tolist(), s["table"].cpu().numpy(), s["path"].cpu().numpy()
    new = []
    for b, m in enumerate(s["path_len"].tolist()):
        pos = ctx[b] + np.arange(m)
        page = torch.from_numpy(table[b, pos // s["page"]].astype(np.int64)).to(DEV)
        slot = torch.from_numpy(pos % s["page"]).to(DEV)
        node = torch.from_numpy((cu[b] + path[b, :m]).astype(np.int64)).to(DEV)
        k[:, page, slot] = s["k_new"][:, node].double()
        v[:, page, slot] = s["v_new"][:, node].double()
        new.append(ctx[b] + m)
    return {"k": k, "v": v, "new_len": np.array(new, dtype=np.int32)}


def _exact_beams(s):
    b, w, v, keep = s["batch"], s["beams"], s["vocab"], s["keep"]
    out = {"scores": np.zeros((b, keep)), "parents": np.zeros((b, keep), np.int32), "tokens": np.zeros((b, keep), np.int32)}
    for i in range(b):
        z = torch.log_softmax(s["logits"][i * w:(i + 1) * w, :v].double(), 1) + s["scores"][i].double()[:, None]
        for j in range(w):
            if s["ended"] is not None and int(s["ended"][i, j]):
                z[j] = -math.inf
                z[j, 0] = float(s["scores"][i, j])
        val, at = torch.sort(z.flatten(), descending=True, stable=True)
        out["scores"][i] = val[:keep].cpu().numpy()
        out["parents"][i], out["tokens"][i] = (at[:keep] // v).cpu().numpy(), (at[:keep] % v).cpu().numpy()
    rows, parent = torch.arange(b, device=DEV)[:, None], torch.from_numpy(out["parents"]).to(DEV).long()
    return {**out, "ids": s["ids"][rows, parent], "hidden": s["hidden"][rows, parent].double()}


_exact = {"attend": _exact_attend, "weigh": _exact_weigh, "evict": _exact_evict, "commit": _exact_commit,
          "beams": _exact_beams}
