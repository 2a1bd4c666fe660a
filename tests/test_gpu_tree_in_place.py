"""Lengths that a call replaces: commitment and eviction with out_len in the
place of the lengths that they read."""
import numpy as np
import pytest

import speculative_decoding_verification_23_gb300 as sv
from test_gpu_tree import i32, make_kv, make_pages, run_evict, same_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("layers,B", [(1, 5), (2, 70), (28, 150), (61, 300)])
def test_commit_over_its_lengths(layers, B):
    rng = np.random.default_rng(layers)
    counts = [int(x) for x in rng.integers(1, 9, B)]
    acc = [int(rng.integers(0, n + 1)) for n in counts]
    ctx = [int(x) for x in rng.integers(0, 60, B)]
    cu = np.concatenate([[0], np.cumsum(counts)])
    table, num = make_pages(rng, [c + n for c, n in zip(ctx, counts)], 16)
    kn, vn = (torch.randn(layers, int(cu[-1]), 2, 64, device="cuda").bfloat16() for _ in range(2))
    path = np.zeros((B, 8), np.int32)
    for b in range(B):
        path[b, :acc[b]] = np.sort(rng.permutation(counts[b])[:acc[b]])
    if B > 5:
        path[3, 0], acc[3] = counts[3], 1      # a node outside its tree
        table[4, 0] = num                       # a page outside the cache
        ctx[4], acc[4] = 0, 1
        ctx[2] = -1
    results = []
    for in_place in (False, True):
        k, v = (torch.zeros(layers, num, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lens = i32(ctx)
        a = sv.make_commit_args(k_new=kn, v_new=vn, cu_nodes=i32(cu), path=i32(path), path_len=i32(acc),
                                cache=sv.make_cache(k, v), block_table=i32(table), ctx_len=lens)
        new_len, st = sv.spec_cache_commit(a, out_len=lens if in_place else None)
        results.append((k, v, new_len, st))
    (k, v, n, st), (k2, v2, n2, st2) = results
    want = [c + m for c, m in zip(ctx, acc)]
    if B > 5:
        want[2] = want[3] = want[4] = -1
        assert st.tolist()[2:5] == [sv.SPEC_STATUS_BAD_LEN, sv.SPEC_STATUS_BAD_LEN, sv.SPEC_STATUS_BAD_PAGE]
    assert n.tolist() == want and n2.tolist() == want and torch.equal(st, st2)
    assert same_bits(k, k2) and same_bits(v, v2)


@pytest.mark.parametrize("lens,keep", [([300, 299, 0, 40], 64), ([3000] * 60 + [3], 500), ([1], 1), ([0], 4)])
def test_eviction_over_its_lengths(lens, keep):
    heads = 8
    rng = np.random.default_rng(keep)
    w = torch.from_numpy(np.exp(rng.standard_normal((len(lens), heads, max(lens) + 3))).astype(np.float32)).cuda()
    results = []
    for in_place in (False, True):
        a, table, to, k, v, k0, v0 = run_evict(w, lens, keep, 0, 0, heads=heads)
        got = sv.spec_cache_evict(a, out_len=a._keep[1] if in_place else None)
        results.append((*got, k, v))
    for x, y in zip(*results):
        assert torch.equal(x, y) if x.dtype != torch.bfloat16 else same_bits(x, y)
    assert results[1][2].tolist() == [min(n, keep) for n in lens] and results[1][3].tolist() == [0] * len(lens)


def test_eviction_of_bad_requests_over_its_lengths():
    w = torch.rand(4, 2, 100, device="cuda")
    a, table, to, k, v, k0, v0 = run_evict(w, [100, 90, 80, 0], 32, 0, 0, break_to=1)
    lens = a._keep[1]
    lens[2] = 101
    index, kept, new_len, st = sv.spec_cache_evict(a, out_len=lens)
    assert new_len.data_ptr() == lens.data_ptr() and new_len.tolist() == [32, -1, -1, 0]
    assert st.tolist() == [0, sv.SPEC_STATUS_BAD_PAGE, sv.SPEC_STATUS_BAD_LEN, 0]
    assert torch.all(index[1:] == -1) and torch.all(kept[1:] == 0)
