"""The operators beside the drafted tree in the order of a serving loop: a round against its plain 64-bit definition,
on another stream, captured into graphs that share a workspace, and the example."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402
import speculative_decoding_verification_23_gb300 as sv  # noqa: E402
from test_gpu_serve import (DEV, DT, Case, commit_args, commit_case, commit_want, gen, i32, normal, same_bytes,  # noqa: E402
                            trees)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Loop:
    """Rounds of a loop: queries and keys turned in place, attention with a window over 16 bits and without one over
    8 bits with one workspace, and both caches' commitment, the lengths in place."""

    def __init__(self, seed, *, dtype="bf16", dim=128, kv=2, group=4, page=16, block=8, ctx=(150, 0, 333), nodes=(9, 5, 17),
                 accepted=(3, 1, 6), window=100, sinks=5, rounds=3):
        rng, g, t = np.random.RandomState(seed), gen(seed), DT[dtype]
        self.dtype, self.page, self.block, self.window, self.sinks = dtype, page, block, window, sinks
        self.start, self.nodes, self.accepted = ctx, nodes, accepted
        need = [-(-(c + rounds * m) // page) for c, m in zip(ctx, accepted)]
        pages, total = sum(need) + 1, sum(nodes)
        ids, at = rng.permutation(pages), 0
        self.tab = np.full((len(ctx), max(need)), -1, np.int32)
        for b, n in enumerate(need):
            self.tab[b, :n] = ids[at:at + n]
            at += n
        self.k, self.v = (normal(g, pages, page, kv, dim, dtype=t) for _ in range(2))
        self.k8, self.v8 = ((60 * torch.randn(pages, page, kv, dim, generator=g, device=DEV)).to(torch.float8_e4m3fn)
                            for _ in range(2))
        self.ks, self.vs = (torch.full((pages, page // block, kv), 2.0 ** -6, device=DEV) for _ in range(2))
        # one projection's queries, keys and values
        self.qkv = normal(g, total, kv * (group + 2), dim, dtype=t, scale=2.0)
        self.q, self.kn, self.vn = self.qkv.split([kv * group, kv, kv], 1)
        self.weight = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(t)
        self.freq = (1e4 ** (-torch.arange(0, dim, 2, device=DEV) / dim)).float()
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.mask = trees(rng, nodes, -(-max(nodes) // 32))
        self.path = np.full((len(ctx), max(accepted)), -1, np.int32)
        for b, (n, m) in enumerate(zip(nodes, accepted)):
            self.path[b, :m] = np.sort(rng.permutation(n)[:m])
        self.pos = np.concatenate([c + np.arange(n) for c, n in zip(ctx, nodes)]).astype(np.int32)
        self.ctx, self.pos_d, cu = i32(ctx), i32(self.pos), i32(self.cu)
        cache, cache8 = sv.make_cache(self.k, self.v), sv.make_cache8(self.k8, self.v8, self.ks, self.vs)
        self.rotate = sv.make_rotate_args(q=self.q, k=self.kn, positions=self.pos_d, inv_freq=self.freq,
                                          q_weight=self.weight, k_weight=self.weight)
        drafted = dict(q=self.q, k_new=self.kn, v_new=self.vn, cu_nodes=cu, max_nodes=max(nodes), block_table=i32(self.tab),
                       ctx_len=self.ctx, tree_mask=torch.from_numpy(self.mask.view(np.int32)).to(DEV))
        self.windowed = sv.make_window_args(cache=cache, window=window, sinks=sinks, **drafted)
        self.attend8 = sv.make_cache8_args(cache=cache8, **drafted)
        commit = dict(k_new=self.kn, v_new=self.vn, cu_nodes=cu, path=i32(self.path), path_len=i32(accepted),
                      block_table=i32(self.tab), ctx_len=self.ctx)
        self.commit = sv.make_commit_args(cache=cache, **commit)
        self.commit8 = sv.make_cache8_commit_args(cache=cache8, **commit)
        self.ws = torch.empty(max(sv.spec_window_workspace_bytes(self.windowed), sv.spec_cache8_workspace_bytes(self.attend8),
                                  256), dtype=torch.uint8, device=DEV)
        shape = self.q.shape
        self.out = [torch.zeros(shape, dtype=t, device=DEV) for _ in range(2)]
        self.lse = [torch.zeros(shape[:2], device=DEV) for _ in range(2)]
        self.status = [i32([9] * len(ctx)) for _ in range(4)]
        self.new_len = i32([0] * len(ctx))

    def attention(self, stream=None):
        for i, (call, a) in enumerate(((sv.spec_window_attention, self.windowed), (sv.spec_cache8_attention, self.attend8))):
            call(a, workspace=self.ws, out=self.out[i], out_lse=self.lse[i], out_status=self.status[i], stream=stream)

    def run(self, stream=None):
        sv.spec_norm_rotate(self.rotate, out_q=self.q, out_k=self.kn, stream=stream)
        self.attention(stream)
        sv.spec_cache_commit(self.commit, out_len=self.new_len, out_status=self.status[2], stream=stream)
        sv.spec_cache8_commit(self.commit8, out_len=self.ctx, out_status=self.status[3], stream=stream)

    def results(self):
        torch.cuda.synchronize()
        return [x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16) if x.element_size() == 2 else
                x.view(torch.int32) for x in (self.qkv, *self.out, *self.lse, self.k, self.v, self.k8, self.v8, self.ks,
                                              self.vs, self.ctx, self.new_len, *self.status)]


def equal(a, b):
    assert all(torch.equal(x, y) for x, y in zip(a.results(), b.results()))
    assert all(int(s.abs().max()) == 0 for s in a.status) and torch.equal(a.ctx, a.new_len)


KINDS = [dict(), dict(dtype="fp16", dim=64, group=7, nodes=(1, 1, 1), accepted=(1, 1, 1)),
         dict(dim=128, kv=1, group=8, page=64, block=64, nodes=(64, 33, 50), accepted=(5, 1, 6), ctx=(700, 40, 64))]


@pytest.mark.parametrize("kw", KINDS)
def test_a_round_against_its_definition(kw):
    a = Loop(1, **kw)
    was = a.qkv.clone()
    pages = [x.clone() for x in (a.k8, a.v8, a.ks, a.vs)]
    a.run()
    torch.cuda.synchronize()
    assert all(int(s.abs().max()) == 0 for s in a.status)
    hq, kv = a.q.shape[1], a.kn.shape[1]
    w = ref.f64(a.weight)
    for x, y in ((was[:, :hq], a.q), (was[:, hq:hq + kv], a.kn)):
        want, tol = ref.rotate(ref.f64(x), w, a.pos, ref.f64(a.freq), float(np.float32(1e-6)), False, a.dtype)
        assert (np.abs(ref.f64(y) - want) <= tol).all()
    assert torch.equal(was[:, hq + kv:], a.vn)
    # the attention of what the rotation gave; commitment wrote past the lengths that it read, except scales of blocks
    # begun before, for which the 8-bit side takes the cache from before
    scale, mask = a.q.shape[2] ** -0.5, a.mask.view(np.int32)
    drafted = [ref.f64(x) for x in (a.q, a.kn, a.vn)]
    k8, v8 = (ref.e4m3(x.view(torch.uint8).cpu().numpy()) for x in pages[:2])
    for i, (k, v, kw2) in enumerate(((ref.f64(a.k), ref.f64(a.v), dict(window=a.window, sinks=a.sinks)),
                                     (k8, v8, dict(scales=[ref.f64(x) for x in pages[2:]], block=a.block)))):
        out, lse, t_out, t_lse = ref.attention(*drafted, a.cu, k, v, a.page, a.tab, a.start, mask, scale, a.dtype, **kw2)
        assert (np.abs(ref.f64(a.lse[i]) - lse) <= t_lse).all() and (np.abs(ref.f64(a.out[i]) - out) <= t_out).all()
    for held, held_scale, x, got, got_scale in ((pages[0], pages[2], a.kn, a.k8, a.ks), (pages[1], pages[3], a.vn, a.v8, a.vs)):
        want, want_scale = ref.commit8(held.view(torch.uint8).cpu().numpy()[None], held_scale.cpu().numpy()[None], ref.f64(x)[None],
                                       a.cu, a.path, a.accepted, a.tab, a.start, a.page, a.block)
        assert same_bytes(got, want[0]) and np.array_equal(got_scale.cpu().numpy(), want_scale[0])
    assert a.ctx.tolist() == [c + m for c, m in zip(a.start, a.accepted)] == a.new_len.tolist()


@pytest.mark.parametrize("kw", KINDS)
def test_another_stream(kw):
    a, b = Loop(2, **kw), Loop(2, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.run()
        b.run(side)
    equal(a, b)


@pytest.mark.parametrize("kw", KINDS)
def test_a_captured_round_replays(kw):
    """The graph reads the lengths at each replay: three rounds, each over a longer text."""
    a, b = Loop(3, **kw), Loop(3, **kw)
    warm = Loop(4, **kw)
    warm.run()                     # loads the kernels before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for _ in range(3):
        a.run()
        graph.replay()
    equal(a, b)
    assert b.ctx.tolist() == [c + 3 * m for c, m in zip(b.start, b.accepted)]


def test_graphs_and_calls_that_share_a_workspace():
    """Two graphs and an eager call use one workspace in turn, in either order, and again after it was overwritten."""
    loops = [Loop(5), Loop(6, **KINDS[2]), Loop(7, dtype="fp16", ctx=(2000, 900, 40))]
    ws = torch.empty(max(x.ws.numel() for x in loops), dtype=torch.uint8, device=DEV)
    for x in loops:
        x.attention()
    torch.cuda.synchronize()
    want = [[y.clone() for y in (*x.out, *x.lse)] for x in loops]
    graphs = []
    for x in loops:
        x.ws = ws
    for x in loops[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.attention()
        graphs.append(g.replay)
    runs = [*graphs, loops[2].attention]
    for order, fill in (((0, 1, 2), 255), ((2, 0, 1), 0), ((1, 1, 0, 2, 0), 127)):
        ws.fill_(fill)
        for x in loops:
            for y in (*x.out, *x.lse):
                y.fill_(-3)
        for i in order:
            runs[i]()
        torch.cuda.synchronize()
        for x, w in zip(loops, want):
            assert all(torch.equal(y, z) for y, z in zip((*x.out, *x.lse), w))


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own."""
    loops = [Loop(8, **KINDS[2]), Loop(9, **KINDS[2])]
    for x in loops:
        x.attention()
    torch.cuda.synchronize()
    want = [[y.clone() for y in (*x.out, *x.lse)] for x in loops]
    sides = [torch.cuda.Stream() for _ in loops]
    for _ in range(20):
        for x, s in zip(loops, sides):
            x.attention(s)
    torch.cuda.synchronize()
    for x, w in zip(loops, want):
        assert all(torch.equal(y, z) for y, z in zip((*x.out, *x.lse), w))


@pytest.mark.parametrize("block", [None, 16])
@pytest.mark.parametrize("nodes", [(0, 2, 0, 1, 0), (0, 40, 0, 64, 0), (0, 0, 0, 0, 0)])
def test_requests_without_nodes(block, nodes):
    """They have no rows and status 0, whatever their lengths; the others are as without them."""
    if not any(nodes):
        c = Case(dtype="bf16", dim=64, kv=1, group=2, page=16, ctx=[40] * 5, nodes=[1] * 5, chain=True, window=None if block else 30,
                 block=block, seed=3)
        a = c.args(q=c.q[:0], k_new=c.k_new[:0], v_new=c.v_new[:0], cu_nodes=i32([0] * 6), max_nodes=0)
        out, lse, status = c.run(a)
        assert out.shape[0] == 0 and status.tolist() == [0] * 5
        return
    c = Case(dtype="bf16", dim=128, kv=2, group=4, page=16, ctx=[600, 77, 0, 1030, 5], nodes=list(nodes), chain=False,
             window=None if block else 200, sinks=0 if block else 3, block=block, seed=3)
    c.check()


def test_results_between_other_rows_and_heads():
    """Results of any strides: what lies between them stays."""
    for block, nodes in ((None, [5, 40]), (16, [5, 40]), (16, [2, 3])):
        c = Case(dtype="bf16", dim=128, kv=2, group=4, page=16, ctx=[130, 700], nodes=nodes, chain=True,
                 window=None if block else 90, block=block, seed=8)
        want, _, _ = c.run()
        big = torch.full((want.shape[0], want.shape[1] + 3, 136), 7.0, dtype=torch.bfloat16, device=DEV)
        out = big[:, 1:-2, :128]
        c.run(out=out)
        assert torch.equal(out, want)
        rest = big.clone()
        rest[:, 1:-2, :128] = 7
        assert (rest == 7).all()


def test_calls_give_the_same_bits_again():
    for kw in KINDS:
        a = Loop(11, **{**kw, "ctx": (3001, 1500, 64)})
        a.attention()
        torch.cuda.synchronize()
        want = [x.clone() for x in (*a.out, *a.lse)]
        for _ in range(5):
            a.attention()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip((*a.out, *a.lse), want))


def test_attention_past_32_bit_offsets():
    """A cache of 5 GB whose last pages hold the text."""
    pages, page, kv, dim = 81920, 64, 8, 128
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    small = Case(dtype="bf16", dim=dim, kv=kv, group=2, page=page, ctx=[300, 500], nodes=[40, 2], chain=True, block=64, seed=5)
    want = small.run()[0]
    k, v = (torch.empty(pages, page, kv, dim, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    ks, vs = (torch.empty(pages, 1, kv, device=DEV) for _ in range(2))
    n = small.k.shape[0]
    for x, y in ((k, small.k), (v, small.v)):
        x[-n:].copy_(y)
    for x, y in ((ks, small.scales[0]), (vs, small.scales[1])):
        x[-n:].copy_(y)
    table = np.where(small.table >= 0, small.table + pages - n, small.table)
    small.k, small.v, small.scales, small.table = k, v, [ks, vs], table
    assert torch.equal(small.run()[0], want)


@pytest.mark.parametrize("B", [31, 257, 700])
def test_commitment_of_many_requests(B):
    """More requests than threads that add them up; some without tokens, some bad."""
    rng = np.random.RandomState(B)
    ctx, nodes = rng.randint(0, 70, B).tolist(), rng.randint(1, 4, B).tolist()
    c = commit_case(dtype="bf16", layers=2, kv=1, dim=64, page=16, block=8, ctx=ctx, nodes=nodes,
                    accepted=[int(rng.randint(0, n + 1)) for n in nodes], seed=B)
    want = commit_want({**c, "m": np.where(np.arange(B) % 7 == 3, 0, c["m"])})
    bad = (np.arange(B) % 7 == 3) & (c["m"] > 0)
    c["path"][bad, 0] = 300      # no such node: nothing of the request is written
    length, status = sv.spec_cache8_commit(commit_args(c))
    assert status.tolist() == np.where(bad, sv.SPEC_STATUS_BAD_LEN, 0).tolist()
    assert length.tolist() == np.where(bad, -1, c["ctx"] + c["m"]).tolist()
    for x, s, (held, scale) in zip((c["k"], c["v"]), (c["ks"], c["vs"]), want):
        assert same_bytes(x, held) and np.array_equal(s.cpu().numpy(), scale)


@pytest.mark.parametrize("dim,group,nodes", [(128, 4, 64), (64, 8, 40), (128, 2, 30), (128, 2, 60), (64, 2, 50), (64, 1, 17)])
def test_many_tiles_give_the_same_bits_again(dim, group, nodes):
    """Dozens of tiles of every CTA, in segments of all lengths, many times."""
    rng, kv, page, B = np.random.RandomState(3), 8, 16, 12
    c = Case(dtype="fp16", dim=dim, kv=kv, group=group, page=page, ctx=rng.randint(1000, 9000, B).tolist(), nodes=[nodes] * B,
             chain=False, block=16, seed=4)
    args = c.args()
    want = c.run(args)
    for _ in range(60):
        assert all(torch.equal(x, y) for x, y in zip(c.run(args), want))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [None, 16, 32])
def test_caches_of_other_layouts(dim, block):
    """A head's tokens side by side; and some heads of a wider cache, whose results are those of a copy of them."""
    kw = dict(dtype="bf16", dim=dim, kv=3, group=4, page=32, ctx=[700, 45, 32], nodes=[9, 17, 1], chain=False,
              window=None if block else 150, sinks=0 if block else 33, block=block, seed=9)
    Case(layout="phsd", **kw).check()
    c = Case(**kw)
    want = c.run()
    wide = [torch.empty(*x.shape[:2], 5, dim, dtype=x.dtype, device=DEV) for x in (c.k, c.v)]
    for w, x in zip(wide, (c.k, c.v)):
        w.view(torch.uint8).fill_(0x7f)     # NaN around them
        w[:, :, 1:4].copy_(x)
    c.k, c.v = (w[:, :, 1:4] for w in wide)
    if block:
        scales = [torch.full((*s.shape[:2], 5), float("nan"), device=DEV) for s in c.scales]
        for w, s in zip(scales, c.scales):
            w[..., 2:5].copy_(s)
        c.scales = [w[..., 2:5] for w in scales]
    assert all(torch.equal(x, y) for x, y in zip(c.run(), want))


def test_queries_and_drafted_tokens_of_one_projection():
    """Strided queries, keys and values, each a part of the same rows."""
    for block, nodes in ((None, [5, 40]), (16, [5, 40]), (16, [2, 3])):
        c = Case(dtype="fp16", dim=128, kv=2, group=4, page=16, ctx=[130, 700], nodes=nodes, chain=True,
                 window=None if block else 90, block=block, seed=12)
        want = c.run()
        rows = torch.full((c.q.shape[0], 13, 128), float("nan"), dtype=torch.float16, device=DEV)
        rows[:, :8], rows[:, 8:10], rows[:, 11:] = c.q, c.k_new, c.v_new
        assert all(torch.equal(x, y) for x, y in zip(c.run(c.args(q=rows[:, :8], k_new=rows[:, 8:10], v_new=rows[:, 11:])), want))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window", [None, 130])
@pytest.mark.parametrize("dim,group,nodes", [(128, 1, (17, 31)), (128, 2, (32, 9)), (64, 1, (33, 64)), (128, 1, (65, 3)),
                                             (64, 2, (64, 33)), (128, 1, (129, 64)), (128, 7, (9, 3))])
def test_numbers_of_rows_over_8_bits(dim, group, nodes, window, dtype):
    """Up to 64 rows a key head, up to 128, and more, of a few tiles and of many that several CTAs share."""
    for ctx in ([130, 257], [6000, 1]):
        Case(dtype=dtype, dim=dim, kv=2, group=group, page=16, ctx=ctx, nodes=list(nodes), chain=False, window=window,
             sinks=3 if window else 0, block=16, seed=sum(nodes) + group).check()


@pytest.mark.parametrize("beams,depth", [(4, 3), (1, 5), (10, 2)])
def test_the_example_of_long_texts(beams, depth):
    import long_text as E

    one = E.generate(seed=1, rounds=40, beams=beams, depth=depth)
    text, lens, held = one
    assert all(n == len(t) - 1 >= 40 for t, n in zip(text, lens))
    # the sinks' page, the window's and those not yet reached
    pages = -(-41 * (depth + 1) // 16)
    assert all(h <= 1 + 3 + pages - n // 16 for h, n in zip(held, lens))
    assert E.generate(seed=1, rounds=40, beams=beams, depth=depth) == one
