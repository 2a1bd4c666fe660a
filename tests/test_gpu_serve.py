"""GPU parity of the operators beside the drafted tree with their plain 64-bit definitions, at sizes and masks where
they can go wrong.  Error bounds are derived in serve_ref.py."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402
import speculative_decoding_verification_23_gb300 as sv  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def normal(g, *shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def trees(rng, counts, words):
    rows = []
    for n in counts:
        seen = []
        for i in range(n):
            m = 1 << i
            if i:
                m |= seen[rng.randint(max(0, i - 6), i)]
            seen.append(m)
        rows += [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in seen]
    return np.array(rows, dtype=np.uint32).reshape(-1, words)


# ---------------------------------------------------- norms and positions

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (64, 64, True), (96, 96, False), (96, 48, True),
                                                 (128, 128, False), (128, 64, False), (128, 8, True), (192, 192, False),
                                                 (192, 64, True), (256, 256, False), (256, 0, False)])
@pytest.mark.parametrize("rows,hq,hk", [(1, 14, 2), (67, 5, 3), (1, 1, 0), (9, 0, 4)])
def test_rotation(dtype, dim, rot, interleaved, rows, hq, hk):
    g = gen(dim + rot + rows)
    t = DT[dtype]
    qkv = normal(g, rows, hq + 2 * hk + 1, dim, dtype=t, scale=3.0)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    wq, wk = normal(g, dim, dtype=t, scale=0.3) + 1, None
    pos = torch.randint(-1000, 1 << 27, (rows,), generator=g, device=DEV, dtype=torch.int32)
    freq = (1e4 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / max(rot, 1))).float()
    a = sv.make_rotate_args(q=q if hq else None, k=k if hk else None, positions=pos, inv_freq=freq,
                            q_weight=wq if hq else None, k_weight=wk, eps=1e-5, interleaved=interleaved)
    got = sv.spec_norm_rotate(a)
    p, f = pos.cpu().numpy(), freq.double().cpu().numpy()
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        if y is None:
            assert x.shape[1] == 0
            continue
        want, tol = ref.rotate(ref.f64(x), None if w is None else ref.f64(w), p, f, float(np.float32(1e-5)), interleaved, dtype)
        assert (np.abs(ref.f64(y) - want) <= tol).all()


def test_rotation_in_place_is_the_same():
    g = gen(5)
    qkv = normal(g, 300, 20, 128, dtype=torch.bfloat16)
    pos = torch.arange(300, dtype=torch.int32, device=DEV) * 977
    freq = (1e6 ** (-torch.arange(0, 128, 2, device=DEV) / 128)).float()
    q, k = qkv[:, :14], qkv[:, 14:17]
    a = sv.make_rotate_args(q=q, k=k, positions=pos, inv_freq=freq)
    out_q, out_k = sv.spec_norm_rotate(a)
    v = qkv[:, 17:].clone()
    sv.spec_norm_rotate(a, out_q=q, out_k=k)
    assert torch.equal(q, out_q) and torch.equal(k, out_k) and torch.equal(qkv[:, 17:], v)


def test_rotation_of_zeros_infinities_and_no_rows():
    freq = torch.ones(32, device=DEV)
    x = torch.zeros(3, 2, 64, dtype=torch.float16, device=DEV)
    x[1, 0, 5], x[2, 1, 3] = float("inf"), float("nan")
    pos = i32([0, 1, 2])
    y, _ = sv.spec_norm_rotate(sv.make_rotate_args(q=x, k=None, positions=pos, inv_freq=freq))
    assert (y[0] == 0).all() and (y[1, 1] == 0).all() and (y[2, 0] == 0).all()
    assert y[1, 0].isnan().any() and y[2, 1].isnan().all()
    y, _ = sv.spec_norm_rotate(sv.make_rotate_args(q=x[:0], k=None, positions=pos[:0], inv_freq=freq))
    assert y.shape == (0, 2, 64)


# --------------------------------------------------------------- attention

class Case:
    """A call of windowed attention or of attention over 8 bits, and its answer."""

    def __init__(self, *, dtype, dim, kv, group, page, ctx, nodes, chain, window=None, sinks=0, block=None, seed=0,
                 zero_scales=False, layout="pshd", bad=None):
        rng, g, t = np.random.RandomState(seed), gen(seed), DT[dtype]
        self.dtype, self.page, self.window, self.sinks, self.block = dtype, page, window, sinks, block
        need = [-(-c // page) for c in ctx]
        width, pages = max(1, max(need)), sum(need) + 2
        ids, at = rng.permutation(pages), 0
        table = np.full((len(ctx), width), -7, np.int32)  # entries past a request's pages are not looked at
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        shape = (pages, page, kv, dim)
        order = {"pshd": (0, 1, 2, 3), "phsd": (0, 2, 1, 3)}[layout]  # how the cache lies in memory
        back = [order.index(i) for i in range(4)]

        def held(x):
            return x.permute(order).contiguous().permute(back)

        if block is None:
            self.k, self.v = (held(normal(g, *shape, dtype=t)) for _ in range(2))
            self.scales = None
        else:
            self.k, self.v = (held((torch.randn(shape, generator=g, device=DEV) * 60).clamp(-448, 448).to(torch.float8_e4m3fn))
                              for _ in range(2))
            sc = [torch.exp(torch.randn(pages, page // block, kv, generator=g, device=DEV)) / 60 for _ in range(2)]
            if zero_scales:
                for s in sc:
                    s[torch.rand(s.shape, generator=g, device=DEV) < 0.4] = 0
            self.scales = sc
        self.counts = nodes
        total = sum(nodes)
        self.q = normal(g, total, kv * group, dim, dtype=t, scale=2.0)
        self.k_new, self.v_new = normal(g, total, kv, dim, dtype=t), normal(g, total, kv, dim, dtype=t)
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.mask = None if chain else trees(rng, nodes, max(1, -(-max(nodes) // 32)))
        self.table, self.ctx = table, np.array(ctx, np.int32)

    def args(self, **kw):
        m = None if self.mask is None else torch.from_numpy(self.mask.view(np.int32)).to(DEV)
        a = dict(q=self.q, k_new=self.k_new, v_new=self.v_new, cu_nodes=i32(self.cu), max_nodes=max(self.counts),
                 block_table=i32(self.table), ctx_len=i32(self.ctx), tree_mask=m)
        a.update(kw)
        if self.block is None:
            return sv.make_window_args(cache=sv.make_cache(self.k, self.v), window=self.window, sinks=self.sinks, **a)
        return sv.make_cache8_args(cache=sv.make_cache8(self.k, self.v, *self.scales), window=self.window or 0,
                                   sinks=self.sinks, **a)

    def run(self, args=None, **kw):
        call = sv.spec_window_attention if self.block is None else sv.spec_cache8_attention
        return call(args or self.args(), **kw)

    def want(self):
        if self.block is None:
            k, v, sc = ref.f64(self.k), ref.f64(self.v), None
        else:
            k, v = (ref.e4m3(x.view(torch.uint8).cpu().numpy()) for x in (self.k, self.v))
            sc = [ref.f64(x) for x in self.scales]
        return ref.attention(ref.f64(self.q), ref.f64(self.k_new), ref.f64(self.v_new), self.cu, k, v, self.page, self.table,
                             self.ctx, None if self.mask is None else self.mask.view(np.int32), self.q.shape[2] ** -0.5,
                             self.dtype, self.window, self.sinks, sc, self.block)

    def check(self, got=None):
        out, lse, status = got or self.run()
        assert status.tolist() == [0] * len(self.ctx)
        w_out, w_lse, t_out, t_lse = self.want()
        o, l = ref.f64(out), ref.f64(lse)
        assert (np.isneginf(l) == np.isneginf(w_lse)).all()
        fine = np.isfinite(w_lse)
        assert (np.abs(l[fine] - w_lse[fine]) <= t_lse[fine]).all(), np.abs(l[fine] - w_lse[fine]).max()
        assert (np.abs(o - w_out) <= t_out).all(), (np.abs(o - w_out) / t_out).max()
        assert (o[~fine] == 0).all()


# both kernels (up to 16 rows a key head, and more), head sizes that only warp tiles take, odd pages
SHAPES = [
    dict(dim=64, kv=2, group=7, page=16, ctx=[1001], nodes=[1], chain=True),
    dict(dim=128, kv=1, group=1, page=16, ctx=[0, 1, 15, 16, 17], nodes=[1, 2, 1, 3, 1], chain=True),
    dict(dim=128, kv=2, group=4, page=16, ctx=[300, 129, 0, 64], nodes=[9, 1, 5, 9], chain=True),
    dict(dim=128, kv=2, group=4, page=32, ctx=[700, 33, 513], nodes=[40, 64, 1], chain=False),
    dict(dim=64, kv=1, group=8, page=64, ctx=[130, 1000], nodes=[64, 33], chain=False),
    dict(dim=96, kv=2, group=3, page=16, ctx=[200, 77], nodes=[7, 2], chain=False),
    dict(dim=192, kv=1, group=2, page=24, ctx=[150, 48], nodes=[5, 12], chain=True),
    dict(dim=256, kv=1, group=5, page=16, ctx=[100], nodes=[20], chain=False),
    dict(dim=128, kv=1, group=4, page=8, ctx=[250, 9], nodes=[17, 3], chain=False, layout="phsd"),
    dict(dim=64, kv=1, group=3, page=5, ctx=[33, 101], nodes=[3, 30], chain=True),
    dict(dim=128, kv=1, group=1, page=128, ctx=[5000], nodes=[150], chain=False),
    dict(dim=128, kv=1, group=2, page=16, ctx=[40, 300], nodes=[256, 200], chain=True),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 4), (64, 0), (100, 1), (256, 20), (4000, 130)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_windows(shape, window, sinks, dtype):
    Case(dtype=dtype, window=window, sinks=sinks, seed=shape, **SHAPES[shape]).check()


def blocks_of(page):
    return sorted({page, 8 if page % 8 == 0 else page, 16 if page % 16 == 0 else 1})


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape,block", [(i, b) for i, s in enumerate(SHAPES) for b in blocks_of(s["page"])])
def test_attention_over_8_bits(shape, block, dtype):
    Case(dtype=dtype, block=block, seed=shape, **SHAPES[shape]).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (6, 3), (100, 1), (300, 140)])
@pytest.mark.parametrize("shape", [0, 2, 3, 4, 5, 8, 11])
def test_windows_over_8_bits(shape, window, sinks, dtype):
    page = SHAPES[shape]["page"]
    Case(dtype=dtype, block=16 if page % 16 == 0 else page, window=window, sinks=sinks, seed=shape, **SHAPES[shape]).check()


@pytest.mark.parametrize("shape", [1, 2, 3, 4])
def test_scales_of_zero(shape):
    Case(dtype="bf16", block=16, zero_scales=True, seed=shape, **SHAPES[shape]).check()


@pytest.mark.parametrize("block", [None, 16])
@pytest.mark.parametrize("nodes", [1, 30])
def test_a_large_window_hides_nothing(block, nodes):
    """With a window over everything the call gives what it gives without one, bit by bit."""
    s = dict(dtype="bf16", dim=128, kv=2, group=4, page=16, ctx=[400, 37], nodes=[nodes, max(1, nodes // 2)], chain=False, seed=3)
    c = Case(window=1 << 30, sinks=7, block=block, **s)
    a = c.run()
    if block is None:
        t = c.args()
        b = sv.spec_tree_attention(sv.make_tree_args(q=c.q, k_new=c.k_new, v_new=c.v_new, cu_nodes=i32(c.cu), max_nodes=nodes,
                                                     cache=sv.make_cache(c.k, c.v), block_table=i32(c.table), ctx_len=i32(c.ctx),
                                                     tree_mask=torch.from_numpy(c.mask.view(np.int32)).to(DEV)))
        assert t.tree.total_nodes == b[0].shape[0]
    else:
        c.window, c.sinks = None, 0
        b = c.run()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("block", [None, 16])
@pytest.mark.parametrize("nodes,chain", [(2, True), (40, False)])
def test_what_a_window_hides_never_reaches(block, nodes, chain):
    """NaN in every hidden slot and in the pages between, whose table entries are no pages: the rows that do not see
    them are as before, and the status is good."""
    s = dict(dtype="bf16", dim=128, kv=2, group=4, page=16, ctx=[1000, 250], nodes=[nodes, nodes], chain=chain, seed=9)
    window, sinks = 100, 20
    c = Case(window=window, sinks=sinks, block=block, **s)
    clean = [x.clone() for x in c.run()]
    for b, n in enumerate(c.ctx):
        for j in range(sinks, n - window):
            page, slot = c.table[b, j // 16], j % 16
            for x in (c.k, c.v):
                (x if block is None else x.view(torch.uint8))[page, slot] = float("nan") if block is None else 0x7f
        for p in range(-(-sinks // 16), (n - window) // 16):
            c.table[b, p] = -1 if p % 2 else 1 << 30
    got = c.run()
    for x, y in zip(clean, got):
        assert torch.equal(x, y)
    # NaN in a value that the first rows of request 0 see and the last ones do not
    j = 1000 - window + 1
    x = c.v if block is None else c.v.view(torch.uint8)
    x[c.table[0, j // 16], j % 16] = float("nan") if block is None else 0x7f
    out, lse, _ = c.run()
    m = None if c.mask is None else c.mask
    for i in range(nodes):
        tree = (np.arange(nodes) <= i) if m is None else ref.bits(m[i].view(np.int32), nodes)
        sees = ref.text(tree, 1000, window, sinks)[j]
        assert bool(out[i].isnan().all()) == bool(sees)
        if not sees:
            assert torch.equal(out[i], clean[0][i])
    assert torch.equal(out[nodes:], clean[0][nodes:]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("block", [None, 16])
@pytest.mark.parametrize("nodes", [2, 40])
def test_masks_that_leave_nothing(block, nodes):
    s = dict(dtype="fp16", dim=64, kv=1, group=4, page=16, ctx=[0, 40], nodes=[nodes, nodes], chain=False, seed=4)
    c = Case(window=30, sinks=0, block=block, **s)
    c.mask[0] = 0
    c.mask[nodes - 1] = 0
    c.mask[nodes + 1] = 0
    c.check()
    out, lse, _ = c.run()
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nodes", [3, 40])
def test_infinities_and_nan_among_drafted_values(dtype, nodes):
    """Over 8 bits: rows that do not see an odd drafted value are as without it; those that do carry it."""
    c = Case(dtype=dtype, dim=128, kv=1, group=4, page=16, ctx=[70], nodes=[nodes], chain=True, block=16, seed=2)
    clean = [x.clone() for x in c.run()]
    c.v_new[1, 0, 7], c.v_new[2, 0, 9] = float("inf"), float("nan")
    out, lse, status = c.run()
    assert status.tolist() == [0] and torch.equal(lse, clean[1]) and torch.equal(out[0], clean[0][0])
    assert (out[1:, :, 7] == math.inf).all() and out[2:, :, 9].isnan().all() and not out[:2, :, 9].isnan().any()


@pytest.mark.parametrize("nodes", [2, 40])
def test_bf16_beyond_the_range_of_fp16(nodes):
    """Queries, drafted keys and values of sizes that fp16 does not have."""
    c = Case(dtype="bf16", dim=128, kv=2, group=4, page=16, ctx=[90, 0], nodes=[nodes, nodes], chain=False, block=16, seed=6)
    c.q.mul_(1e-20)
    c.k_new.mul_(1e20)
    c.v_new.mul_(1e25)
    for s in c.scales:
        s.mul_(1e15)
    c.check()
    c = Case(dtype="bf16", dim=64, kv=1, group=4, page=16, ctx=[33], nodes=[nodes], chain=False, block=16, seed=7)
    c.q.mul_(1e9)
    c.k_new.mul_(1e-9)
    c.v_new.mul_(1e-12)
    for i, s in enumerate(c.scales):
        s.mul_(1e-9 if i == 0 else 1e-12)
    c.check()


@pytest.mark.parametrize("block", [None, 16])
@pytest.mark.parametrize("nodes", [2, 40])
def test_bad_lengths_and_pages(block, nodes):
    s = dict(dtype="bf16", dim=128, kv=2, group=4, page=16, ctx=[100, 60, 500, 32], nodes=[nodes] * 4, chain=True, seed=8)
    c = Case(window=90, sinks=3, block=block, **s)
    clean = c.run()[0].clone()
    c.ctx[1] = c.table.shape[1] * 16 + 1   # past its table
    c.table[2, 30] = c.k.shape[0]          # within the window
    out, lse, status = c.run()
    assert status.tolist() == [0, sv.SPEC_STATUS_BAD_LEN, sv.SPEC_STATUS_BAD_PAGE, 0]
    for b in (1, 2):
        assert out[b * nodes:(b + 1) * nodes].isnan().all() and lse[b * nodes:(b + 1) * nodes].isnan().all()
    for b in (0, 3):
        assert torch.equal(out[b * nodes:(b + 1) * nodes], clean[b * nodes:(b + 1) * nodes])


@pytest.mark.parametrize("block", [None, 16])
def test_a_long_context_is_split(block):
    c = Case(dtype="bf16", dim=128, kv=1, group=2, page=64, ctx=[9000, 3], nodes=[10, 2], chain=False, block=block,
             window=8000, sinks=70, seed=11)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,nodes", [(128, 4, 64), (64, 8, 40), (128, 2, 30)])
def test_many_tiles_over_8_bits(dtype, dim, group, nodes):
    """Dozens of tiles of each CTA, of many segments: as the 16-bit kernel over the same values, up to the rounding of
    weights in both (half a step relative to what they add up, and of the result) and of the keys and values to bf16
    (exact: e4m3 with scales of powers of two)."""
    g, rng, t = gen(3), np.random.RandomState(3), DT[dtype]
    kv, page, B = 8, 16, 12
    ctx = rng.randint(1000, 9000, B).tolist()
    need = [-(-c // page) for c in ctx]
    table = np.zeros((B, max(need)), np.int32)
    ids, at = rng.permutation(sum(need)), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    shape = (sum(need), page, kv, dim)
    k8, v8 = ((torch.randn(shape, generator=g, device=DEV) * 64).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (2.0 ** torch.randint(-7, -4, (sum(need), 1, kv), generator=g, device=DEV) for _ in range(2))
    q = normal(g, B * nodes, kv * group, dim, dtype=t, scale=0.7)
    k_new, v_new = normal(g, B * nodes, kv, dim, dtype=t), normal(g, B * nodes, kv, dim, dtype=t)
    m = torch.from_numpy(trees(rng, [nodes] * B, -(-nodes // 32)).view(np.int32)).to(DEV)
    a = dict(q=q, k_new=k_new, v_new=v_new, cu_nodes=i32(np.arange(B + 1) * nodes), max_nodes=nodes, block_table=i32(table),
             ctx_len=i32(ctx), tree_mask=m)
    out, lse, status = sv.spec_cache8_attention(sv.make_cache8_args(cache=sv.make_cache8(k8, v8, ks, vs), **a))
    k16, v16 = ((x.float() * s[..., None]).to(t) for x, s in ((k8, ks), (v8, vs)))
    want, w_lse, _ = sv.spec_tree_attention(sv.make_tree_args(cache=sv.make_cache(k16, v16), **a))
    assert status.tolist() == [0] * B
    # softmax weights over at least 1000 keys of values up to 14 in size
    assert (lse - w_lse).abs().max() <= 1e-4
    assert (out.float() - want.float()).abs().max() <= (2 * 2.0 ** -8 + 2.0 ** -10 if dtype == "bf16" else 4 * 2.0 ** -11) * 2.0
    again = sv.spec_cache8_attention(sv.make_cache8_args(cache=sv.make_cache8(k8, v8, ks, vs), **a))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_few_requests_rows_and_layers_of_an_8_bit_cache():
    """Layers, a cache of other strides, outputs of other strides; a request without nodes."""
    g = gen(1)
    layers, pages, page, kv, dim = 3, 9, 16, 2, 64
    store = (torch.randn(pages, layers, 2, kv, page, dim, generator=g, device=DEV) * 60).to(torch.float8_e4m3fn)
    k, v = (store[:, :, i].permute(1, 0, 3, 2, 4) for i in range(2))
    scales = torch.rand(2, kv, pages, layers, 1, generator=g, device=DEV) / 60
    ks, vs = (scales[i].permute(2, 1, 3, 0) for i in range(2))
    cache = sv.make_cache8(k, v, ks, vs)
    c = Case(dtype="fp16", dim=dim, kv=kv, group=2, page=page, ctx=[50, 17, 20], nodes=[3, 0, 2], chain=True, block=16, seed=2)
    for layer in range(layers):
        a = sv.make_cache8_args(
            q=c.q, k_new=c.k_new, v_new=c.v_new, cu_nodes=i32(c.cu), max_nodes=3, cache=cache, block_table=i32(c.table),
            ctx_len=i32(c.ctx), layer=layer)
        wide = torch.zeros(5, 10, dim, dtype=torch.float16, device=DEV)
        got = sv.spec_cache8_attention(a, out=wide[:, 3:7])
        c.k, c.v, c.scales = k[layer], v[layer], [ks[layer], vs[layer]]
        c.check(got)
        assert (wide[:, :3] == 0).all() and (wide[:, 7:] == 0).all()


# -------------------------------------------------------------- commitment

def commit_case(*, dtype, layers, kv, dim, page, block, ctx, nodes, accepted, seed, odd=False, sizes=True):
    rng, g, t = np.random.RandomState(seed), gen(seed), DT[dtype]
    need = [-(-(c + m) // page) for c, m in zip(ctx, accepted)]
    pages = sum(need) + 1
    ids, at = rng.permutation(pages), 0
    table = np.full((len(ctx), max(1, max(need))), -3, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    k, v = ((torch.randn(layers, pages, page, kv, dim, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            for _ in range(2))
    ks, vs = (torch.exp(2 * torch.randn(layers, pages, page // block, kv, generator=g, device=DEV)) / 128 for _ in range(2))
    total = sum(nodes)
    k_new, v_new = (torch.randn(layers, total, kv, dim, generator=g, device=DEV) for _ in range(2))
    if sizes:
        for x in (k_new, v_new):
            x.mul_(torch.exp(3 * torch.randn(layers, total, kv, 1, generator=g, device=DEV)))
    k_new, v_new = k_new.to(t), v_new.to(t)
    if odd:
        k_new[0, 0, 0, 3], v_new[-1, -1, -1, 0], v_new[0, 1, 0, 1] = float("inf"), float("nan"), -float("inf")
        k_new[:, 2] = 0
    path = np.full((len(ctx), max(1, max(accepted))), -1, np.int32)
    for b, (n, m) in enumerate(zip(nodes, accepted)):
        path[b, :m] = rng.permutation(n)[:m]
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    return dict(k=k, v=v, ks=ks, vs=vs, k_new=k_new, v_new=v_new, path=path, m=np.array(accepted, np.int32), cu=cu,
                table=table, ctx=np.array(ctx, np.int32), page=page, block=block)


def commit_args(c, ctx=None):
    return sv.make_cache8_commit_args(k_new=c["k_new"], v_new=c["v_new"], cu_nodes=i32(c["cu"]), path=i32(c["path"]),
                                      path_len=i32(c["m"]), cache=sv.make_cache8(c["k"], c["v"], c["ks"], c["vs"]),
                                      block_table=i32(c["table"]), ctx_len=i32(c["ctx"]) if ctx is None else ctx)


def commit_want(c):
    return [ref.commit8(x.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), ref.f64(n), c["cu"], c["path"], c["m"], c["table"],
                        c["ctx"], c["page"], c["block"]) for x, s, n in ((c["k"], c["ks"], c["k_new"]), (c["v"], c["vs"], c["v_new"]))]


def same_bytes(got, want):
    """Equal bytes; a NaN is a NaN of either sign."""
    g = got.view(torch.uint8).cpu().numpy()
    return ((g == want) | ((g & 127 == 127) & (want & 127 == 127))).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kw", [
    dict(layers=3, kv=2, dim=64, page=16, block=16, ctx=[777], nodes=[9], accepted=[4]),
    dict(layers=2, kv=3, dim=128, page=32, block=16, ctx=[0, 5, 16, 31, 40], nodes=[33, 20, 1, 3, 9], accepted=[33, 17, 1, 2, 0]),
    dict(layers=1, kv=1, dim=96, page=8, block=8, ctx=[3, 8], nodes=[30, 9], accepted=[30, 9]),
    dict(layers=2, kv=2, dim=192, page=24, block=24, ctx=[30], nodes=[50], accepted=[50]),
    dict(layers=1, kv=2, dim=256, page=64, block=64, ctx=[10, 65], nodes=[200, 3], accepted=[150, 3]),
    dict(layers=1, kv=1, dim=128, page=256, block=256, ctx=[100, 0], nodes=[700, 300], accepted=[700, 300]),
    dict(layers=2, kv=1, dim=64, page=10, block=5, ctx=[7], nodes=[40], accepted=[21]),
    dict(layers=1, kv=1, dim=128, page=7, block=1, ctx=[7], nodes=[20], accepted=[11]),
])
@pytest.mark.parametrize("odd", [False, True])
def test_commitment_to_8_bits(kw, dtype, odd):
    c = commit_case(dtype=dtype, seed=kw["dim"] + kw["page"], odd=odd, **kw)
    want = commit_want(c)
    new_len, status = sv.spec_cache8_commit(commit_args(c))
    assert status.tolist() == [0] * len(kw["ctx"]) and new_len.tolist() == (c["ctx"] + c["m"]).tolist()
    for x, s, (wx, ws) in ((c["k"], c["ks"], want[0]), (c["v"], c["vs"], want[1])):
        assert (s.cpu().numpy() == ws).all()
        assert same_bytes(x, wx)


def test_commitment_in_place_of_the_lengths():
    c = commit_case(dtype="bf16", layers=5, kv=2, dim=64, page=16, block=16, ctx=[20, 3], nodes=[9, 5], accepted=[6, 5], seed=1)
    want = commit_want(c)
    ctx = i32(c["ctx"])
    new_len, status = sv.spec_cache8_commit(commit_args(c, ctx), out_len=ctx)
    assert new_len is ctx and ctx.tolist() == [26, 8] and status.tolist() == [0, 0]
    assert same_bytes(c["k"], want[0][0]) and same_bytes(c["v"], want[1][0])


@pytest.mark.parametrize("accepted", [[6, 5, 4, 300], [6, 5, 4, 7]])
@pytest.mark.parametrize("what", ["page", "node", "negative", "length", "offsets"])
def test_commitment_of_a_bad_request(what, accepted):
    """Nothing of a bad request is written, and the others are as they should be."""
    nodes = [9, 8, 7, 310]
    c = commit_case(dtype="fp16", layers=2, kv=2, dim=64, page=16, block=16, ctx=[20, 14, 60, 5], nodes=nodes, accepted=accepted, seed=3)
    want = commit_want({**c, "m": np.array([c["m"][0], 0, c["m"][2], c["m"][3]], np.int32)})
    status = sv.SPEC_STATUS_BAD_LEN
    if what == "page":
        c["table"][1, 1] = c["k"].shape[1]
        status = sv.SPEC_STATUS_BAD_PAGE
    elif what == "node":
        c["path"][1, 4] = 8
    elif what == "negative":
        c["m"][1] = -1
    elif what == "length":
        c["ctx"][1] = c["table"].shape[1] * 16 - 2
    else:
        c["m"][1] = c["path"].shape[1] + 1
    new_len, got = sv.spec_cache8_commit(commit_args(c))
    assert got.tolist() == [0, status, 0, 0] and new_len.tolist()[1] == -1
    assert (c["ks"].cpu().numpy() == want[0][1]).all() and same_bytes(c["k"], want[0][0]) and same_bytes(c["v"], want[1][0])


def test_commitment_past_32_bit_offsets():
    """A cache of more than 2^32 bytes: its last page is written, its first is not."""
    pages, page, kv, dim = 2200, 1024, 16, 128
    k = torch.zeros(pages, page, kv, dim, dtype=torch.float8_e4m3fn, device=DEV)
    v = torch.zeros_like(k)
    sc = [torch.zeros(pages, 8, kv, device=DEV) for _ in range(2)]
    cache = sv.make_cache8(k, v, *sc)
    x = torch.randn(3, kv, dim, device=DEV).bfloat16()
    table = i32([[0, pages - 1]])
    a = sv.make_cache8_commit_args(k_new=x, v_new=x, cu_nodes=i32([0, 3]), path=i32([[2, 0, 1]]), path_len=i32([3]), cache=cache,
                                   block_table=table, ctx_len=i32([page]))
    new_len, status = sv.spec_cache8_commit(a)
    assert status.tolist() == [0] and new_len.tolist() == [page + 3]
    assert not k[0].view(torch.uint8).any() and not sc[0][0].any()
    for i, n in enumerate([2, 0, 1]):
        got = k[pages - 1, i].float() * sc[0][pages - 1, 0][:, None]
        assert (got - x[n].float()).abs().max() <= 2.0 ** -4 * x[n].float().abs().max()
    q = torch.randn(1, kv, dim, device=DEV).bfloat16()
    out, _, status = sv.spec_cache8_attention(sv.make_cache8_args(
        q=q, k_new=x[:1], v_new=x[:1], cu_nodes=i32([0, 1]), max_nodes=1, cache=cache, block_table=table, ctx_len=new_len,
        window=4))
    kk = torch.cat([k[pages - 1, :3].float() * sc[0][pages - 1, 0][:, None], x[:1].float()])
    vv = torch.cat([v[pages - 1, :3].float() * sc[1][pages - 1, 0][:, None], x[:1].float()])
    p = torch.softmax(torch.einsum("hd,khd->hk", q[0].float(), kk) * dim ** -0.5, 1)
    want = torch.einsum("hk,khd->hd", p, vv)
    assert status.tolist() == [0] and (out[0].float() - want).abs().max() <= 2.0 ** -7 * vv.abs().max()
