"""Results over what a call reads are refused on the host: nothing is
enqueued, and no buffer changes."""
import numpy as np
import pytest

import speculative_decoding_verification_23_gb300 as sv
from test_gpu_tree import Tree, i32, run_evict

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def refused(call, *buffers):
    was = [b.clone() for b in buffers]
    with pytest.raises(sv.SpecError) as e:
        call()
    assert e.value.code == sv.SPEC_ERR_SHAPE
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(was, buffers))


def test_beams():
    z = torch.randn(12, 1000, device="cuda").bfloat16()
    both = torch.zeros(2 * 12, device="cuda")
    cum, ended = both[:12].view(3, 4), torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    a = sv.make_beam_args(logits=z, V=1000, scores=cum, keep=4, finished=ended)
    refused(lambda: sv.spec_beam_select(a, out_scores=cum), both, ended)
    refused(lambda: sv.spec_beam_select(a, out_scores=both[8:20].view(3, 4)), both, ended)
    refused(lambda: sv.spec_beam_select(a, out_parents=ended), both, ended)
    refused(lambda: sv.spec_beam_select(a, out_tokens=ended), both, ended)
    refused(lambda: sv.spec_beam_select(a, out_status=ended.view(-1)[9:]), both, ended)
    refused(lambda: sv.spec_beam_select(a, out_tokens=z.view(-1)[3000:3024].view(torch.int32).view(3, 4)), both)
    s, p, t, st = sv.spec_beam_select(a, out_scores=both[12:].view(3, 4))  # beside them is no overlap
    assert st.tolist() == [0] * 3 and torch.all(cum == 0)


def test_lengths_and_weights():
    w = torch.rand(2, 2, 100, device="cuda")
    a, table, to, k, v, k0, v0 = run_evict(w, [100, 90], 32, 0, 0)
    lens, from_table, to_table = a._keep[1], a._keep[3], a._keep[4]
    part = w.view(-1)[200:328].view(2, 2, 32)
    refused(lambda: sv.spec_cache_evict(a, out_kept=part), w, lens)
    refused(lambda: sv.spec_cache_evict(a, out_status=lens), w, lens)
    refused(lambda: sv.spec_cache_evict(a, out_len=from_table.view(-1)[:2]), from_table, lens)
    refused(lambda: sv.spec_cache_evict(a, out_len=to_table.view(-1)[:2]), to_table, lens)
    four = i32([100, 90, 7, 7])
    b = sv.make_evict_args(weights=w, kv_len=four[:2], keep=32, cache=a._keep[2], block_table=from_table,
                           to_table=to_table)
    refused(lambda: sv.spec_cache_evict(b, out_len=four[1:3]), four)   # over a part of them


def test_paths():
    k, v = (torch.zeros(3, 8, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    new = torch.ones(3, 6, 2, 64, dtype=torch.bfloat16, device="cuda")
    ints = i32([5, 6, 1, 2, 0, 3, 6, 9])
    ctx, length, cu = ints[:2], ints[2:4], ints[4:7]
    path, table = i32([[0, 2], [0, 1]]), i32([[0, 1], [2, 3]])
    a = sv.make_commit_args(k_new=new, v_new=new, cu_nodes=cu, path=path, path_len=length, cache=sv.make_cache(k, v),
                            block_table=table, ctx_len=ctx)
    for out in (length, ints[1:3], cu[:2], path.view(-1)[2:], table.view(-1)[:2]):
        refused(lambda: sv.spec_cache_commit(a, out_len=out), ints, path, table, k, v)
    refused(lambda: sv.spec_cache_commit(a, out_status=ctx), ints, k, v)
    assert sv.spec_cache_commit(a, out_len=ctx)[0].tolist() == [6, 8]


def test_attention_and_its_weights():
    t = Tree(3, [4, 2], [40, 70], 4, 2, 64, 16)
    a = t.args()
    refused(lambda: sv.spec_tree_attention(a, out_status=t.ctx_d), t.ctx_d, t.table_d)
    refused(lambda: sv.spec_tree_attention(a, out_status=t.cu_d[1:]), t.ctx_d, t.cu_d)
    out, lse, st = sv.spec_tree_attention(a)
    rows = torch.zeros(2 * 2 * 80 + 40, device="cuda")
    rows[2 * 2 * 80 - 4:2 * 2 * 80 + 20] = lse.view(-1)
    w = sv.make_weigh_args(q=t.q, lse=rows[316:340].view(6, 4), cu_rows=t.cu_d, max_rows=4, cache=t.cache,
                           block_table=t.table_d, kv_len=t.ctx_d)
    refused(lambda: sv.spec_attention_weights(w, out=rows[:320].view(2, 2, 80)), rows)
    refused(lambda: sv.spec_attention_weights(w, ld=80, out_status=t.ctx_d), rows, t.ctx_d)
    old = torch.zeros(321, device="cuda")
    refused(lambda: sv.spec_attention_weights(w, old[:320].view(2, 2, 80), out=old[1:].view(2, 2, 80)), old)
    assert sv.spec_attention_weights(w, old[:320].view(2, 2, 80), out=old[:320].view(2, 2, 80))[1].tolist() == [0, 0]
