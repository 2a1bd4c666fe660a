"""The drafted-tree operators against plain 64-bit implementations, at the
sizes, layouts and masks where they can go wrong."""
import numpy as np
import pytest

import speculative_decoding_verification_23_gb300 as sv
import tree_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make_pages(rng, lens, page, spare=3):
    """A table of scattered pages; its unused entries point outside."""
    need = [-(-n // page) for n in lens]
    num = sum(need) + spare
    ids = rng.permutation(num)[:sum(need)]
    table = np.full((len(lens), max(1, max(need))), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, num


def make_kv(rng, num, page, heads, dim, dtype, layout="slots", layers=None, layer=0):
    """Key and value tensors [.., pages, page, heads, dim] full of NaN, in a layout."""
    shape = {"slots": (num, page, heads, dim), "heads": (num, heads, page, dim)}[layout]
    if layers:
        shape = (layers, *shape)
    out = []
    for _ in range(2):
        t = torch.full(shape, float("nan"), dtype=TYPES[dtype], device="cuda")
        out.append(t if layout == "slots" else t.transpose(-3, -2))
    return out


def fill(t, rng, table, lens, page):
    """Normal values in the slots in use of t [pages, page, heads, dim]; returns the whole as float64."""
    for b, n in enumerate(lens):
        pos = np.arange(n)
        x = torch.from_numpy(rng.standard_normal((n, *t.shape[2:])).astype(np.float32)).to(t.device, t.dtype)
        if n:
            t[torch.from_numpy(table[b, pos // page].astype(np.int64)).cuda(),
              torch.from_numpy(pos % page).cuda()] = x
    return R.f64(t)


def random_masks(rng, counts, words):
    rows = []
    for n in counts:
        seen = []
        for i in range(n):
            seen.append((1 << i) | (seen[rng.integers(max(0, i - 6), i)] if i else 0))
        rows += [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in seen]
    return np.array(rows, dtype=np.uint32).reshape(-1, words)


class Tree:
    """One attention call's inputs, on the device and in 64 bits."""

    def __init__(self, seed, counts, ctx, heads_q, heads, dim, page, dtype="bf16", masks="random", layout="slots",
                 layers=None, layer=0, strided=False, q_scale=2.0, max_nodes=None):
        rng = np.random.default_rng(seed)
        self.rng, self.page, self.dtype, self.ctx, self.counts = rng, page, dtype, list(ctx), list(counts)
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
        total = int(self.cu[-1])
        self.max_nodes = max_nodes or max(1, max(counts))
        self.table, num = make_pages(rng, ctx, page)
        k, v = make_kv(rng, num, page, heads, dim, dtype, layout, layers)
        self.k_all, self.v_all = k, v
        kl, vl = (k[layer], v[layer]) if layers else (k, v)
        self.k64, self.v64 = fill(kl, rng, self.table, ctx, page), fill(vl, rng, self.table, ctx, page)

        def packed(h, scale=1.0):
            wide = h + 2 if strided else h
            t = torch.from_numpy((scale * rng.standard_normal((total, wide, dim))).astype(np.float32))
            t = t.to("cuda", TYPES[dtype])
            return t[:, 1:1 + h] if strided else t

        self.q, self.kn, self.vn = packed(heads_q, q_scale), packed(heads), packed(heads)
        words = -(-self.max_nodes // 32)
        self.mask = None
        if isinstance(masks, str):
            self.mask = random_masks(rng, counts, words)
        elif masks is not None:
            self.mask = np.asarray(masks, dtype=np.uint32).reshape(total, words)
        self.scale, self.layer = dim ** -0.5, layer

    def args(self, **kw):
        self.cache = sv.make_cache(self.k_all, self.v_all)
        mask = None if self.mask is None else torch.from_numpy(self.mask.view(np.int32)).cuda()
        self.table_d, self.ctx_d, self.cu_d = i32(self.table), i32(self.ctx), i32(self.cu)
        return sv.make_tree_args(q=self.q, k_new=self.kn, v_new=self.vn, cu_nodes=self.cu_d, max_nodes=self.max_nodes,
                                 cache=self.cache, block_table=self.table_d, ctx_len=self.ctx_d, tree_mask=mask,
                                 layer=self.layer, **kw)

    def reference(self):
        return R.attention(R.f64(self.q), R.f64(self.kn), R.f64(self.vn), self.cu, self.k64, self.v64, self.page,
                           self.table, self.ctx, self.mask, self.scale, self.dtype)

    def check(self, out, lse, status):
        o, e, ot, et = self.reference()
        got, gl = R.f64(out), R.f64(lse)
        assert np.array_equal(status.cpu().numpy(), np.zeros(len(self.ctx), np.int32))
        assert np.array_equal(np.isneginf(gl), np.isneginf(e))
        fin = np.isfinite(e)
        assert np.all(np.abs(gl[fin] - e[fin]) <= et[fin]), np.max(np.abs(gl[fin] - e[fin]) / et[fin])
        assert np.array_equal(np.isnan(got), np.isnan(o))
        odd = ~np.isfinite(o)
        assert np.array_equal(got[odd & ~np.isnan(o)], o[odd & ~np.isnan(o)])
        assert np.all(np.isfinite(got[~odd]))
        d = np.abs(got[~odd] - o[~odd])
        assert np.all(d <= ot[~odd]), np.max(d / ot[~odd])


SHAPES = [
    # counts, ctx, heads_q, heads, dim, page, dtype
    ([1], [0], 4, 2, 64, 16, "bf16"),
    ([1], [1], 4, 2, 64, 16, "fp16"),
    ([1], [1001], 14, 2, 64, 16, "bf16"),
    ([1, 1, 1], [63, 64, 65], 8, 8, 128, 16, "bf16"),
    ([5, 0, 1, 17], [0, 40, 127, 300], 14, 2, 64, 16, "bf16"),
    ([9, 2, 5], [128, 129, 255], 28, 4, 128, 16, "fp16"),
    ([16], [2000], 28, 4, 128, 16, "bf16"),
    ([64, 33], [511, 1030], 8, 2, 128, 64, "bf16"),
    ([129], [70], 4, 2, 128, 32, "bf16"),
    ([256], [300], 2, 1, 64, 32, "fp16"),
    ([40], [1500], 32, 4, 128, 64, "bf16"),
    ([7], [130], 3, 1, 96, 16, "bf16"),
    ([6, 3], [77, 260], 5, 1, 192, 8, "fp16"),
    ([12], [333], 8, 2, 256, 16, "bf16"),
    ([8, 4], [90, 200], 6, 2, 128, 1, "bf16"),
    ([8, 4], [90, 200], 6, 2, 64, 3, "bf16"),
    ([20], [500], 8, 2, 128, 24, "fp16"),
    ([20], [500], 8, 2, 128, 8, "bf16"),
    ([18], [900], 16, 2, 128, 256, "bf16"),
    ([3] * 40, list(range(0, 400, 10)), 4, 2, 64, 16, "bf16"),
]


@pytest.mark.parametrize("counts,ctx,hq,h,dim,page,dtype", SHAPES)
@pytest.mark.parametrize("masks", [None, "random"])
def test_attention_matches_the_definition(counts, ctx, hq, h, dim, page, dtype, masks):
    t = Tree(len(counts) + dim + page, counts, ctx, hq, h, dim, page, dtype, masks)
    t.check(*sv.spec_tree_attention(t.args()))


@pytest.mark.parametrize("layout,layers,layer,strided", [("heads", None, 0, False), ("slots", 3, 1, False),
                                                         ("heads", 2, 1, True), ("slots", None, 0, True)])
@pytest.mark.parametrize("hq", [4, 28])
def test_attention_layouts(layout, layers, layer, strided, hq):
    t = Tree(3, [9, 20], [100, 257], hq, 4, 128, 16, "bf16", "random", layout, layers, layer, strided)
    out = torch.empty(29, hq + 3, 128, dtype=torch.bfloat16, device="cuda").fill_(7.0)
    t.check(*sv.spec_tree_attention(t.args(), out=out[:, 2:2 + hq]))
    assert torch.all(out[:, :2] == 7.0) and torch.all(out[:, 2 + hq:] == 7.0)


@pytest.mark.parametrize("hq,dim", [(2, 64), (16, 128)])
def test_rows_that_see_nothing_are_zero(hq, dim):
    counts = [5, 12]
    masks = np.zeros((17, 1), np.uint32)
    masks[1] = 0x3
    masks[6] = 0xFFFFF000  # bits past the tree
    masks[10] = 0xFFFFFFFF
    t = Tree(5, counts, [0, 0], hq, 2, dim, 16, "bf16", masks)
    out, lse, st = sv.spec_tree_attention(t.args())
    t.check(out, lse, st)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0])) and torch.all(out[6] == 0)
    # the same over some cached tokens: the cached ones alone
    t = Tree(5, counts, [33, 200], hq, 2, dim, 16, "bf16", masks)
    t.check(*sv.spec_tree_attention(t.args()))


@pytest.mark.parametrize("hq,dim,dtype", [(2, 64, "bf16"), (16, 128, "bf16"), (16, 128, "fp16"), (4, 256, "bf16")])
def test_what_a_row_does_not_see_does_not_reach_it(hq, dim, dtype):
    counts, n = [20], 20
    t = Tree(6, counts, [150], hq, 2, dim, 16, dtype)
    # node 4 holds NaN and infinities; of the others only node 9 sees it
    for i in range(n):
        t.mask[i] &= ~np.uint32(1 << 4)
    t.mask[9] |= np.uint32(1 << 4)
    t.kn[4] = 0.0
    t.vn[4] = 1.0
    t.vn[4, 0, 0], t.vn[4, 0, 1], t.vn[4, 1, 2] = float("nan"), float("inf"), float("-inf")
    out, lse, st = sv.spec_tree_attention(t.args())
    t.check(out, lse, st)
    assert torch.isnan(out[9, 0, 0]) and torch.isposinf(out[9, 0, 1]) and torch.isneginf(out[9, hq // 2, 2])
    # and in the keys, seen by nobody
    t.mask[9] &= ~np.uint32(1 << 4)
    t.kn[4] = float("nan")
    t.check(*sv.spec_tree_attention(t.args()))


def test_a_seen_infinity_in_the_cache_is_an_infinity():
    t = Tree(8, [3], [70], 4, 2, 64, 16)
    t.v_all[int(t.table[0, 1]), 2, 0, 5] = float("inf")
    t.v64 = R.f64(t.v_all)
    out, lse, st = sv.spec_tree_attention(t.args())
    t.check(out, lse, st)
    assert torch.all(torch.isposinf(out[:, :2, 5]))


def test_large_logits_move_the_reference():
    t = Tree(9, [10], [700], 8, 2, 128, 16, "bf16", q_scale=30.0)
    t.check(*sv.spec_tree_attention(t.args()))
    # ascending logits: the running maximum moves in every tile
    t = Tree(10, [4], [900], 4, 2, 64, 16, "bf16", None)
    ramp = torch.linspace(-4, 4, 900, device="cuda")
    for j in range(900):
        t.k_all[int(t.table[0, j // 16]), j % 16] = ramp[j].to(torch.bfloat16)
    t.q[:] = 1.5
    t.k64 = R.f64(t.k_all)
    t.check(*sv.spec_tree_attention(t.args()))


def test_a_long_context_is_split_and_joined():
    t = Tree(11, [2], [20011], 14, 2, 64, 16)
    t.check(*sv.spec_tree_attention(t.args()))
    t = Tree(12, [24], [9001], 8, 2, 128, 64, "fp16")
    t.check(*sv.spec_tree_attention(t.args()))


def test_many_requests_of_many_lengths():
    rng = np.random.default_rng(1)
    counts, ctx = rng.integers(0, 12, 200), rng.integers(0, 90, 200)
    t = Tree(13, counts, ctx, 4, 1, 64, 16, max_nodes=16)
    t.check(*sv.spec_tree_attention(t.args()))


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements, its last pages in use."""
    page, heads, dim = 16, 8, 128
    num = (1 << 31) // (page * heads * dim) + 64
    k = torch.zeros(num, page, heads, dim, dtype=torch.bfloat16, device="cuda")
    t = Tree(14, [3], [40], 16, 8, dim, page)
    big = t.table.copy()
    big[0, :3] = [num - 1, 5, num - 7]
    for i in range(3):
        k[int(big[0, i])] = t.k_all[int(t.table[0, i])]
    small_k, small_v, small_table = t.k64, t.v64, t.table
    t.v_all = t.k_all
    t.v64 = t.k64
    want = t.reference()
    t.k_all = t.v_all = k
    t.table = big
    out, lse, st = sv.spec_tree_attention(t.args())
    assert np.all(np.abs(R.f64(out) - want[0]) <= want[2])


def test_bad_lengths_and_pages_are_reported():
    t = Tree(15, [4, 5, 3, 6], [100, 200, 50, 300], 28, 4, 128, 16)
    want = t.reference()
    t.table[1, 7] = 1 << 20      # outside the cache
    t.table[3, 2] = -1
    t.ctx[2] = -5
    out, lse, st = sv.spec_tree_attention(t.args())
    assert st.tolist() == [0, sv.SPEC_STATUS_BAD_PAGE, sv.SPEC_STATUS_BAD_LEN, sv.SPEC_STATUS_BAD_PAGE]
    assert np.all(np.abs(R.f64(out)[:4] - want[0][:4]) <= want[2][:4])
    assert torch.all(torch.isnan(out[4:])) and torch.all(torch.isnan(lse[4:]))
    t.ctx[2] = 10 ** 6           # past the table
    out, lse, st = sv.spec_tree_attention(t.args())
    assert st.tolist()[2] == sv.SPEC_STATUS_BAD_LEN and torch.all(torch.isnan(out[9:12]))


def test_streams_graphs_and_workspaces():
    t = Tree(16, [9, 17], [900, 33], 28, 4, 128, 16)
    a = t.args()
    ws = sv.make_tree_workspace(a)
    ws.random_(0, 256)
    out, lse, st = sv.spec_tree_attention(a, workspace=ws)
    again = sv.spec_tree_attention(a, workspace=ws)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sv.spec_tree_attention(a, stream=side)
    side.synchronize()
    assert torch.equal(out, other[0])
    buf = torch.zeros_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_tree_attention(a, workspace=ws, out=buf, out_lse=lse, out_status=st)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf, out)
    t.q.mul_(-0.5)
    g.replay()
    torch.cuda.synchronize()
    t.check(buf, lse, st)


# ------------------------------------------------------- attention weights

@pytest.mark.parametrize("rows,lens,hq,h,dim,page,dtype", [
    ([1], [1], 4, 2, 64, 16, "bf16"),
    ([5], [4001], 28, 4, 128, 16, "bf16"),
    ([1, 0, 9, 3], [64, 65, 200, 3], 14, 2, 64, 16, "fp16"),
    ([40], [300], 8, 2, 128, 24, "bf16"),
    ([6, 6], [6, 130], 4, 4, 96, 3, "bf16"),
    ([33], [129], 3, 1, 192, 8, "fp16"),
    ([10], [500], 4, 2, 256, 1, "bf16"),
    ([300], [700], 2, 1, 64, 64, "bf16"),
])
@pytest.mark.parametrize("with_before", [False, True])
def test_weights_match_the_definition(rows, lens, hq, h, dim, page, dtype, with_before):
    rng = np.random.default_rng(dim + len(rows))
    table, num = make_pages(rng, lens, page)
    k, _ = make_kv(rng, num, page, h, dim, dtype, "heads")
    k64 = fill(k, rng, table, lens, page)
    cu = np.concatenate([[0], np.cumsum(rows)])
    q = torch.from_numpy((2 * rng.standard_normal((cu[-1], hq, dim))).astype(np.float32)).to("cuda", TYPES[dtype])
    ld = max(lens) + 5
    lse = torch.from_numpy(rng.uniform(1, 6, (cu[-1], hq)).astype(np.float32)).cuda()
    if cu[-1] > 3:
        lse[2, 0] = float("inf")  # a row that adds nothing
    before = torch.from_numpy(rng.uniform(0, 9, (len(rows), h, ld)).astype(np.float32)).cuda() if with_before else None
    a = sv.make_weigh_args(q=q, lse=lse, cu_rows=i32(cu), max_rows=max(rows), cache=sv.make_cache(k, k),
                           block_table=i32(table), kv_len=i32(lens))
    out, st = sv.spec_attention_weights(a, before, ld=ld)
    want, tol = R.weights(R.f64(q), R.f64(lse), cu, k64, page, table, lens, dim ** -0.5,
                          None if before is None else R.f64(before), ld)
    assert st.tolist() == [0] * len(rows)
    d = np.abs(R.f64(out) - want)
    assert np.all(d <= tol), np.max(d / np.maximum(tol, 1e-300))
    if with_before:  # in place
        keep = out.clone()
        sv.spec_attention_weights(a, before, out=before)
        assert torch.equal(before, keep)


def test_the_weights_of_a_row_add_up_to_one():
    t = Tree(17, [5], [700], 28, 4, 128, 16, "bf16", None)
    out, lse, st = sv.spec_tree_attention(t.args())
    # the drafted tokens accepted as they are: written to the cache, then weighed
    lens = [705]
    table = np.concatenate([t.table, np.full((1, 1), t.k_all.shape[0] - 1, np.int32)], 1)
    free = [p for p in range(t.k_all.shape[0]) if p not in t.table[0, :44]]
    table[0, 43:45] = [t.table[0, 43], free[0]]
    c = sv.make_commit_args(k_new=t.kn, v_new=t.vn, cu_nodes=t.cu_d, path=i32([[0, 1, 2, 3, 4]]), path_len=i32([5]),
                            cache=t.cache, block_table=i32(table), ctx_len=t.ctx_d)
    new_len, st = sv.spec_cache_commit(c)
    assert new_len.tolist() == lens and st.tolist() == [0]
    w, st = sv.spec_attention_weights(
        sv.make_weigh_args(q=t.q, lse=lse, cu_rows=t.cu_d, max_rows=5, cache=t.cache, block_table=i32(table),
                           kv_len=i32(lens)), ld=705)
    total = w.double().sum(2).cpu().numpy()
    assert np.all(np.abs(total - 5 * 7) < 35 * 705 * 2.0 ** -22)


def test_weights_report_bad_requests():
    rng = np.random.default_rng(2)
    lens = [50, 60, 70, 20]
    table, num = make_pages(rng, lens, 16)
    k, _ = make_kv(rng, num, 16, 2, 64, "bf16")
    fill(k, rng, table, lens, 16)
    table[1, 2] = num
    cu = [0, 2, 4, 6, 8]
    q = torch.randn(8, 4, 64, device="cuda").bfloat16()
    lse = torch.zeros(8, 4, device="cuda")
    a = sv.make_weigh_args(q=q, lse=lse, cu_rows=i32(cu), max_rows=2, cache=sv.make_cache(k, k),
                           block_table=i32(table), kv_len=i32([50, 60, 500, 1]))
    out, st = sv.spec_attention_weights(a, ld=80)
    assert st.tolist() == [0, sv.SPEC_STATUS_BAD_PAGE, sv.SPEC_STATUS_BAD_LEN, sv.SPEC_STATUS_BAD_LEN]
    assert torch.all(torch.isfinite(out[0])) and torch.all(torch.isnan(out[2:]))
    # keys do not depend on one another: those of the bad page alone
    assert torch.all(torch.isnan(out[1, :, 32:48])) and torch.all(torch.isfinite(out[1, :, :32]))
    assert torch.all(torch.isfinite(out[1, :, 48:60])) and torch.all(out[1, :, 60:] == 0)


# ---------------------------------------------------------------- eviction

def run_evict(w, lens, keep, sink, recent, page=16, heads=2, dim=64, dtype="bf16", layout="slots", break_to=None):
    rng = np.random.default_rng(len(lens) + keep)
    table, num = make_pages(rng, lens, page, spare=0)
    m = [min(n, keep) for n in lens]
    to, more = make_pages(rng, m, page, spare=1)
    ld_to = -(-keep // page)
    to = np.concatenate([np.where(to < 1 << 30, to + num, to),
                         np.full((len(lens), max(0, ld_to - to.shape[1])), 1 << 30, np.int32)], 1).astype(np.int32)
    if break_to is not None:
        to[break_to, 0] = num + more
    k, v = make_kv(rng, num + more, page, heads, dim, dtype, layout)
    fill(k, rng, table, lens, page)
    fill(v, rng, table, lens, page)
    k0, v0 = k.clone(), v.clone()
    a = sv.make_evict_args(weights=w, kv_len=i32(lens), keep=keep, sink=sink, recent=recent, cache=sv.make_cache(k, v),
                           block_table=i32(table), to_table=i32(to))
    return a, table, to, k, v, k0, v0


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("lens,keep,sink,recent,page,dim,layout", [
    ([100], 32, 4, 8, 16, 64, "slots"),
    ([1], 1, 0, 0, 16, 64, "slots"),
    ([0, 5, 64, 65], 64, 2, 3, 16, 64, "heads"),
    ([300, 299], 100, 60, 40, 24, 96, "slots"),      # nothing left to choose
    ([40000], 1000, 4, 128, 64, 128, "slots"),
    ([17000, 90], 333, 0, 0, 3, 192, "slots"),
    ([500], 499, 0, 1, 1, 256, "heads"),
])
@pytest.mark.parametrize("kind", ["tail", "ties", "equal", "odd"])
def test_eviction_keeps_the_largest(lens, keep, sink, recent, page, dim, layout, kind):
    rng = np.random.default_rng(keep)
    ld = max(lens) + 3
    w = np.exp(2 * rng.standard_normal((len(lens), 2, ld))).astype(np.float32)
    if kind == "ties":
        w = np.floor(w).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":
        w -= 1.0
        w[:, :, ::7] = np.nan
        w[:, :, 1::11] = -np.inf
        w[:, :, 2::13] = np.inf
        w[:, :, 3::17] = -0.0
        w[:, :, 4::19] = 0.0
    wt = torch.from_numpy(w).cuda()
    a, table, to, k, v, k0, v0 = run_evict(wt, lens, keep, sink, recent, page, 2, dim, layout=layout)
    index, kept, new_len, st = sv.spec_cache_evict(a)
    assert st.tolist() == [0] * len(lens) and new_len.tolist() == [min(n, keep) for n in lens]
    k1, v1 = k0.clone(), v0.clone()
    for b, n in enumerate(lens):
        for h in range(2):
            wi, wk = R.evict(w[b, h], n, keep, sink, recent)
            assert np.array_equal(index[b, h].cpu().numpy(), wi)
            assert np.array_equal(kept[b, h].cpu().numpy(), wk, equal_nan=True)
            m = min(n, keep)
            src, dst = wi[:m].astype(np.int64), np.arange(m)
            sp, dp = torch.from_numpy(table[b, src // page].astype(np.int64)).cuda(), torch.from_numpy(
                to[b, dst // page].astype(np.int64)).cuda()
            ss, ds = torch.from_numpy(src % page).cuda(), torch.from_numpy(dst % page).cuda()
            k1[dp, ds, h], v1[dp, ds, h] = k0[sp, ss, h], v0[sp, ss, h]
    assert same_bits(k, k1) and same_bits(v, v1)


def test_eviction_moves_nothing_of_a_bad_request():
    lens = [100, 90, 80]
    w = torch.rand(3, 2, 100, device="cuda")
    a, table, to, k, v, k0, v0 = run_evict(w, lens, 32, 0, 0, break_to=1)
    table[2, 1] = -3
    a2 = sv.make_evict_args(weights=w, kv_len=i32([100, 90, 80]), keep=32, cache=sv.make_cache(k, v),
                            block_table=i32(table), to_table=i32(to))
    index, kept, new_len, st = sv.spec_cache_evict(a2)
    assert st.tolist() == [0, sv.SPEC_STATUS_BAD_PAGE, sv.SPEC_STATUS_BAD_PAGE] and new_len.tolist() == [32, -1, -1]
    assert torch.all(index[1:] == -1) and torch.all(kept[1:] == 0)
    used = torch.from_numpy(to[0, :2].astype(np.int64)).cuda()
    keepers = torch.ones(k.shape[0], dtype=torch.bool, device="cuda")
    keepers[used] = False
    assert same_bits(k[keepers], k0[keepers]) and same_bits(v[keepers], v0[keepers])
    a3 = sv.make_evict_args(weights=w, kv_len=i32([101, -1, 99]), keep=32, cache=sv.make_cache(k, v),
                            block_table=i32(table), to_table=i32(to))
    assert sv.spec_cache_evict(a3)[3].tolist()[:2] == [sv.SPEC_STATUS_BAD_LEN] * 2


# ---------------------------------------------------------- the path

@pytest.mark.parametrize("layers,page,dim,layout", [(1, 16, 64, "slots"), (5, 16, 128, "heads"), (3, 3, 96, "slots"),
                                                    (2, 1, 256, "slots"), (28, 64, 128, "slots")])
def test_commit_writes_the_path_and_nothing_else(layers, page, dim, layout):
    rng = np.random.default_rng(layers)
    counts, ctx, acc = [9, 1, 0, 33, 5], [100, 0, 7, 15, 16], [4, 1, 0, 17, 0]
    cu = np.concatenate([[0], np.cumsum(counts)])
    table, num = make_pages(rng, [c + m for c, m in zip(ctx, acc)], page)
    k, v = make_kv(rng, num, page, 2, dim, "bf16", layout, layers)
    k0, v0 = k.clone(), v.clone()
    kn = torch.randn(layers, cu[-1], 2, dim, device="cuda").bfloat16()
    vn = torch.randn(layers, cu[-1], 2, dim, device="cuda").bfloat16()
    path = np.full((5, 20), -1, np.int32)
    for b in range(5):
        path[b, :acc[b]] = np.sort(rng.permutation(counts[b])[:acc[b]])
    a = sv.make_commit_args(k_new=kn, v_new=vn, cu_nodes=i32(cu), path=i32(path), path_len=i32(acc),
                            cache=sv.make_cache(k, v), block_table=i32(table), ctx_len=i32(ctx))
    new_len, st = sv.spec_cache_commit(a)
    assert st.tolist() == [0] * 5 and new_len.tolist() == [c + m for c, m in zip(ctx, acc)]
    for b in range(5):
        for i in range(acc[b]):
            pos = ctx[b] + i
            k0[:, int(table[b, pos // page]), pos % page] = kn[:, cu[b] + path[b, i]]
            v0[:, int(table[b, pos // page]), pos % page] = vn[:, cu[b] + path[b, i]]
    assert same_bits(k, k0) and same_bits(v, v0)


def test_commit_refuses_bad_requests_whole():
    k = torch.zeros(8, 16, 2, 64, dtype=torch.float16, device="cuda")
    v = k.clone()
    kn = torch.ones(12, 2, 64, dtype=torch.float16, device="cuda")
    table = np.array([[0, 1], [2, 9], [4, 5], [6, 7]], np.int32)
    a = sv.make_commit_args(k_new=kn, v_new=kn, cu_nodes=i32([0, 3, 6, 9, 12]),
                            path=i32([[0, 2], [0, 1], [0, 3], [0, 1]]), path_len=i32([2, 2, 2, 3]),
                            cache=sv.make_cache(k, v), block_table=i32(table), ctx_len=i32([3, 15, 3, 3]))
    new_len, st = sv.spec_cache_commit(a)
    bad = sv.SPEC_STATUS_BAD_LEN
    assert st.tolist() == [0, sv.SPEC_STATUS_BAD_PAGE, bad, bad] and new_len.tolist() == [5, -1, -1, -1]
    assert int((k != 0).sum()) == 2 * 2 * 64 and torch.all(k[2:] == 0)


# ------------------------------------------------------------------- beams

def check_beams(z, V, cum, keep, ended=None, end_token=0):
    B, W = cum.shape
    s, p, t, st = sv.spec_beam_select(sv.make_beam_args(logits=z, V=V, scores=cum, keep=keep, finished=ended,
                                                        end_token=end_token))
    assert st.tolist() == [0] * B
    z64, c64 = R.f64(z[:, :V]).reshape(B, W, V), R.f64(cum)
    e = None if ended is None else ended.cpu().numpy()
    for b in range(B):
        ws, wp, wt, gap = R.beams(z64[b], c64[b], None if e is None else e[b], end_token, keep)
        gs, gp, gt = s[b].double().cpu().numpy(), p[b].cpu().numpy(), t[b].cpu().numpy()
        assert np.array_equal(np.isneginf(gs), np.isneginf(ws))
        fin = np.isfinite(ws)
        # a row's sum errs by 2^-21 (its exponentials) and the score by its rounding
        assert np.all(np.abs(gs[fin] - ws[fin]) <= 2.0 ** -20 + np.abs(ws[fin]) * 2.0 ** -24)
        # two scores nearer than that may change places, unless they are of one beam or the same
        near = (gap > 0) & (gap < 2.0 ** -19)
        if not near.any():
            assert np.array_equal(gp, wp) and np.array_equal(gt, wt)
        else:
            assert len(set(zip(gp.tolist(), gt.tolist())) - set(zip(wp.tolist(), wt.tolist()))) <= near.sum()


@pytest.mark.parametrize("B,W,keep,V,dtype", [
    (1, 1, 1, 1, "fp32"), (1, 1, 4, 3, "bf16"), (2, 3, 5, 7, "fp32"), (1, 4, 4, 151936, "bf16"),
    (5, 2, 64, 1001, "bf16"), (3, 64, 64, 257, "fp32"), (2, 8, 8, 50257, "bf16"), (40, 3, 7, 4099, "fp32"),
    (1, 64, 33, 8193, "bf16"), (1, 1, 64, 152064, "fp32"), (700, 1, 2, 300, "bf16"),
])
def test_beams_match_the_definition(B, W, keep, V, dtype):
    g = torch.Generator(device="cuda").manual_seed(V + keep)
    z = (3 * torch.randn(B * W, V + (-V) % 8, generator=g, device="cuda")).to(TYPES[dtype])
    z[:, V:] = float("nan")
    cum = -4 * torch.rand(B, W, generator=g, device="cuda")
    check_beams(z, V, cum, keep)
    ended = (torch.rand(B, W, generator=g, device="cuda") < 0.4).int()
    z2 = z.clone()
    z2[ended.flatten().bool()] = float("nan")  # not read
    check_beams(z2, V, cum, keep, ended, V - 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_beam_ties_go_to_the_lowest(dtype):
    V = 9000
    z = torch.zeros(4, V, dtype=TYPES[dtype], device="cuda")
    cum = torch.zeros(1, 4, device="cuda")
    s, p, t, st = sv.spec_beam_select(sv.make_beam_args(logits=z, V=V, scores=cum, keep=64))
    assert t[0].tolist() == list(range(64)) and p[0].tolist() == [0] * 64
    cum[0, 2] = 1.0
    z[2, 5000:] = 1.0
    s, p, t, st = sv.spec_beam_select(sv.make_beam_args(logits=z, V=V, scores=cum, keep=64))
    assert t[0].tolist() == list(range(5000, 5064)) and p[0].tolist() == [2] * 64
    # few distinct values, so that most places are ties
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randint(-2, 3, (6, V), generator=g, device="cuda").to(TYPES[dtype])
    check_beams(z, V, torch.tensor([[0.0, -1.5, -0.25], [0.0, -3.0, -0.5]], device="cuda"), 40)


@pytest.mark.parametrize("W,keep,V", [(7, 18, 2075), (2, 64, 300), (1, 64, 70), (3, 33, 9001), (8, 64, 152064)])
@pytest.mark.parametrize("allowed", [3, 40, 5000])
def test_constrained_vocabularies(W, keep, V, allowed):
    """Most tokens masked by the lowest finite value, fewer allowed than are kept, or not by much."""
    for dtype in (torch.float32, torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(V + allowed)
        z = torch.full((2 * W, V + (-V) % 8), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        at = torch.randperm(V, generator=g, device="cuda")[:allowed]
        z[:, at] = (2 * torch.randn(2 * W, len(at), generator=g, device="cuda")).to(dtype)
        check_beams(z, V, -2 * torch.rand(2, W, generator=g, device="cuda"), keep)
        z[z == torch.finfo(dtype).min] = float("-inf")
        check_beams(z, V, -2 * torch.rand(2, W, generator=g, device="cuda"), keep)


def test_masked_logits_and_dead_beams():
    V, inf = 5000, float("inf")
    g = torch.Generator(device="cuda").manual_seed(4)
    z = torch.full((6, V), -inf, device="cuda")
    z[0, 4000] = 1.0
    z[1, 17:20] = torch.tensor([-900.0, -901.0, -900.0], device="cuda")  # far below, the whole of its row
    z[3] = torch.randn(V, generator=g, device="cuda")
    z[4] = torch.finfo(torch.float32).min
    cum = torch.tensor([[0.0, -1.0, -2.0], [-inf, -0.5, -inf]], device="cuda")
    z[3] = float("nan")  # a dead beam's logits are not read
    check_beams(z, V, cum, 6)


def test_beams_report_bad_logits():
    for dtype in (torch.float32, torch.bfloat16):
        z = torch.randn(6, 4096, device="cuda").to(dtype)
        z[1, 4095] = float("nan")
        z[4, 7] = float("inf")
        cum = torch.zeros(3, 2, device="cuda")
        s, p, t, st = sv.spec_beam_select(sv.make_beam_args(logits=z, V=4096, scores=cum, keep=3))
        assert st.tolist() == [sv.SPEC_STATUS_BAD_LOGITS, 0, sv.SPEC_STATUS_BAD_LOGITS]
        assert torch.all(t[0] == -1) and torch.all(torch.isneginf(s[2])) and torch.all(p[1] >= 0)
        cum[1, 0] = float("nan")
        assert sv.spec_beam_select(sv.make_beam_args(logits=z, V=4096, scores=cum, keep=3))[3].tolist()[1] != 0


def test_beam_calls_repeat_and_replay():
    z = torch.randn(16, 30000, device="cuda").bfloat16()
    cum = -torch.rand(4, 4, device="cuda")
    a = sv.make_beam_args(logits=z, V=30000, scores=cum, keep=5)
    ws = sv.make_beam_workspace(a)
    ws.random_(0, 256)
    first = [x.clone() for x in sv.spec_beam_select(a, workspace=ws)]
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, sv.spec_beam_select(a, workspace=ws)))
    bufs = [torch.zeros_like(x) for x in first]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_beam_select(a, workspace=ws, out_scores=bufs[0], out_parents=bufs[1], out_tokens=bufs[2],
                            out_status=bufs[3])
    for _ in range(3):
        for x in bufs:
            x.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, bufs))


@pytest.mark.parametrize("shape,dtype,lead", [((7,), torch.uint8, None), ((33, 3), torch.int32, None),
                                              ((896,), torch.bfloat16, 3), ((5, 2, 64), torch.float16, 2),
                                              ((40001,), torch.float32, None), ((1,), torch.int64, None), ((0,), torch.int32, None)])
def test_reordering(shape, dtype, lead):
    B, W, K = 5, 4, 6
    full = (*((lead,) if lead else ()), B, W, *shape)
    src = torch.randint(0, 100, full, device="cuda").to(dtype)
    parents = torch.randint(0, W, (B, K), device="cuda", dtype=torch.int32)
    parents[2, 3] = -1
    dst = torch.full((*((lead,) if lead else ()), B, K, *shape), 77, device="cuda").to(dtype)
    small = torch.arange(B * W, device="cuda", dtype=torch.int32).view(B, W)
    small_dst = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    sv.spec_beam_reorder(sv.make_reorder_args(parents=parents, beams=W, states=[(src, dst), (small, small_dst)]))
    rows = torch.arange(B, device="cuda")[:, None]
    at = parents.clamp(min=0).long()
    want = src[:, rows, at] if lead else src[rows, at]
    (want[:, 2, 3] if lead else want[2, 3]).zero_()
    assert torch.equal(dst, want)
    ws = small[rows, at]
    ws[2, 3] = 0
    assert torch.equal(small_dst, ws)


def test_reordering_of_views():
    base = torch.randn(6, 5, 9, 30, device="cuda")
    src = base[:, :, 2:6]                     # [6, 5, 4, 30]: outer 6, B 5, W 4
    dst = torch.zeros(6, 5, 8, 31, device="cuda")[:, :, ::2, :30]
    parents = torch.randint(0, 4, (5, 4), device="cuda", dtype=torch.int32)
    sv.spec_beam_reorder(sv.make_reorder_args(parents=parents, beams=4, states=[(src, dst)]))
    assert torch.equal(dst, src[:, torch.arange(5, device="cuda")[:, None], parents.long()])
