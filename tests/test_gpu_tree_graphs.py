"""Commitment, weights, eviction and reordering captured into a graph, on
another stream, and over a cache whose offsets pass 32 bits."""
import numpy as np
import pytest

import speculative_decoding_verification_23_gb300 as sv
import tree_ref as R
from test_gpu_tree import Tree, i32, make_pages, same_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


class Loop:
    """A round of a serving loop after its attention: commit, weigh, evict, reorder, each into buffers of its own."""

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.lens, self.acc, self.n = [150, 70, 333], [3, 1, 5], [5, 2, 5]
        after = [a + m for a, m in zip(self.lens, self.acc)]
        table, num = make_pages(rng, after, 16)
        to, more = make_pages(rng, [64] * 3, 16, spare=0)
        to = np.where(to < 1 << 30, to + num, to).astype(np.int32)
        g = torch.Generator(device="cuda").manual_seed(seed)

        def bf16(*shape):
            return torch.randn(shape, generator=g, device="cuda").bfloat16()

        self.k, self.v = (bf16(2, num + more, 16, 2, 128) for _ in range(2))
        self.k_new, self.v_new = bf16(2, 12, 2, 128), bf16(2, 12, 2, 128)
        self.q, self.lse = bf16(9, 8, 128), 5 + torch.rand(9, 8, generator=g, device="cuda")
        self.cache = sv.make_cache(self.k, self.v)
        path = np.zeros((3, 5), np.int32)
        for b in range(3):
            path[b, :self.acc[b]] = np.sort(rng.permutation(self.n[b])[:self.acc[b]])
        self.ctx, self.new_len = i32(self.lens), i32([0] * 3)
        self.weights = torch.rand(3, 2, 360, generator=g, device="cuda")
        self.commit = sv.make_commit_args(k_new=self.k_new, v_new=self.v_new, cu_nodes=i32([0, 5, 7, 12]),
                                          path=i32(path), path_len=i32(self.acc), cache=self.cache,
                                          block_table=i32(table), ctx_len=self.ctx)
        self.weigh = sv.make_weigh_args(q=self.q, lse=self.lse, cu_rows=i32([0, 3, 4, 9]), max_rows=5, cache=self.cache,
                                        block_table=i32(table), kv_len=self.new_len, layer=1)
        self.evict = sv.make_evict_args(weights=self.weights, kv_len=self.new_len, keep=64, sink=4, recent=16, layer=1,
                                        cache=self.cache, block_table=i32(table), to_table=i32(to))
        self.parents = i32(rng.integers(-1, 4, (3, 4)))
        self.state = torch.randint(0, 1000, (3, 4, 77), generator=g, device="cuda", dtype=torch.int32)
        self.order = torch.zeros_like(self.state)
        self.reorder = sv.make_reorder_args(parents=self.parents, beams=4, states=[(self.state, self.order)])
        self.index = torch.zeros(3, 2, 64, dtype=torch.int32, device="cuda")
        self.kept = torch.zeros(3, 2, 64, device="cuda")
        self.short, self.status = i32([0] * 3), [i32([9] * 3) for _ in range(3)]

    def run(self, stream=None):
        sv.spec_cache_commit(self.commit, out_len=self.new_len, out_status=self.status[0], stream=stream)
        sv.spec_attention_weights(self.weigh, self.weights, out=self.weights, out_status=self.status[1], stream=stream)
        sv.spec_cache_evict(self.evict, out_index=self.index, out_kept=self.kept, out_len=self.short,
                            out_status=self.status[2], stream=stream)
        sv.spec_beam_reorder(self.reorder, stream=stream)

    def results(self):
        torch.cuda.synchronize()
        return [self.k, self.v, self.weights, self.index, self.kept, self.short, self.new_len, self.order, *self.status]


def equal(a, b):
    assert all(same_bits(x, y) if x.dtype == torch.bfloat16 else torch.equal(x, y)
               for x, y in zip(a.results(), b.results()))
    assert all(int(s.abs().max()) == 0 for s in a.status)


def test_another_stream():
    a, b = Loop(1), Loop(1)
    a.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.run(side)
    side.synchronize()
    equal(a, b)


def test_replays():
    a, b = Loop(2), Loop(2)
    held = [x.clone() for x in b.results()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    equal_start = all(torch.equal(x, y) for x, y in zip(held[2:8], b.results()[2:8]))
    assert equal_start  # a capture computes nothing
    a.run()
    g.replay()
    equal(a, b)
    for x in (a, b):  # other inputs in the same buffers
        x.k_new.mul_(-2)
        x.q.mul_(0.5)
        x.ctx.copy_(i32([140, 76, 300]))
        x.parents.copy_(i32([[0, 0, 1, 3], [2, 2, -1, 1], [3, 2, 1, 0]]))
    a.run()
    g.replay()
    equal(a, b)


def test_replays_in_place():
    """Lengths that grow with every replay."""
    a, b = Loop(3), Loop(3)
    for x in (a, b):
        x.commit_lens = i32([100, 20, 30])
    commits = []
    for x in (a, b):
        args = sv.SpecCommitArgs.from_buffer_copy(x.commit)
        args.ctx_len = x.commit_lens.data_ptr()
        commits.append(args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_cache_commit(commits[1], out_len=b.commit_lens, out_status=b.status[0])
    for step in range(1, 5):
        sv.spec_cache_commit(commits[0], out_len=a.commit_lens, out_status=a.status[0])
        g.replay()
        torch.cuda.synchronize()
        want = [100 + 3 * step, 20 + step, 30 + 5 * step]
        assert a.commit_lens.tolist() == want and b.commit_lens.tolist() == want
        assert same_bits(a.k, b.k) and same_bits(a.v, b.v)


@pytest.fixture(scope="module")
def big():
    """Keys of more than 2^31 elements; their last pages are in use."""
    num = (1 << 31) // (16 * 8 * 128) + 64
    return torch.zeros(num, 16, 8, 128, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("hq", [16, 64])  # warp tiles, and tensor memory
def test_attention_past_32_bits(big, hq):
    t = Tree(14, [3], [40], hq, 8, 128, 16)
    num = big.shape[0]
    at = t.table.copy()
    at[0, :3] = [num - 1, 5, num - 7]
    for i in range(3):
        big[int(at[0, i])] = t.k_all[int(t.table[0, i])]
    t.v_all, t.v64 = t.k_all, t.k64
    want, lse, tol, lse_tol = t.reference()
    t.k_all = t.v_all = big
    t.table = at
    out, got, st = sv.spec_tree_attention(t.args())
    assert st.tolist() == [0]
    assert np.all(np.abs(R.f64(out) - want) <= tol) and np.all(np.abs(R.f64(got) - lse) <= lse_tol)


@pytest.mark.parametrize("rows", [3, 80])  # 6 and 160 rows per key head on tensor memory; more on warps below
@pytest.mark.parametrize("warp", [False, True])
def test_weights_past_32_bits(big, rows, warp):
    rng = np.random.default_rng(rows)
    num, n = big.shape[0], 90
    table = np.array([[num - 1, 5, num - 7, num - 30, 9, num - 12]], np.int32)
    big[torch.from_numpy(table[0].astype(np.int64)).cuda()] = torch.from_numpy(
        rng.standard_normal((6, 16, 8, 128)).astype(np.float32)).cuda().bfloat16()
    hq = 32 if warp and rows == 80 else 16
    q = torch.from_numpy(rng.standard_normal((rows, hq, 128)).astype(np.float32)).cuda().bfloat16()
    lse = torch.from_numpy(rng.uniform(1, 6, (rows, hq)).astype(np.float32)).cuda()
    small = big[torch.from_numpy(table[0].astype(np.int64)).cuda()]
    want, tol = R.weights(R.f64(q), R.f64(lse), [0, rows], R.f64(small), 16, np.arange(6, dtype=np.int32)[None], [n],
                          128 ** -0.5, None, 96)
    # more rows than tensor memory keeps take the other kernel
    a = sv.make_weigh_args(q=q, lse=lse, cu_rows=i32([0, rows]), max_rows=300 if warp else rows,
                           cache=sv.make_cache(big, big), block_table=i32(table), kv_len=i32([n]))
    out, st = sv.spec_attention_weights(a, ld=96)
    assert st.tolist() == [0] and np.all(np.abs(R.f64(out) - want) <= tol)


def test_paths_and_eviction_past_32_bits(big):
    num = big.shape[0]
    table, to = [[num - 1, 5, num - 7]], [[num - 3, num - 40]]
    new = torch.randn(20, 8, 128, device="cuda").bfloat16()
    big[torch.tensor(table[0], device="cuda")] = torch.randn(3, 16, 8, 128, device="cuda").bfloat16()
    a = sv.make_commit_args(k_new=new, v_new=new, cu_nodes=i32([0, 20]), path=i32([[1, 4, 19]]), path_len=i32([3]),
                            cache=sv.make_cache(big, big), block_table=i32(table), ctx_len=i32([38]))
    n, st = sv.spec_cache_commit(a)
    assert n.tolist() == [41] and st.tolist() == [0]
    assert same_bits(big[num - 7, 6:9], new[[1, 4, 19]])
    w = torch.rand(1, 8, 41, device="cuda")
    rows = big[torch.tensor(table[0], device="cuda")].flatten(0, 1)[:41].clone()
    e = sv.make_evict_args(weights=w, kv_len=n, keep=20, cache=sv.make_cache(big, big), block_table=i32(table),
                           to_table=i32(to))
    index, kept, m, st = sv.spec_cache_evict(e)
    assert m.tolist() == [20] and st.tolist() == [0]
    got = big[torch.tensor(to[0], device="cuda")].flatten(0, 1)[:20]
    want = torch.stack([rows[index[0, h].long(), h] for h in range(8)], 1)
    assert same_bits(got, want)
    assert torch.equal(index[0].long().sort(1).values, w[0].topk(20, 1).indices.sort(1).values)
