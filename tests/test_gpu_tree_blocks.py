"""One argument block of attention weights, two threads, two row lengths."""
import threading

import pytest

import speculative_decoding_verification_23_gb300 as sv
from test_gpu_tree import i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_threads_share_a_block():
    lens = [70, 33]
    k = torch.randn(8, 16, 2, 64, device="cuda").bfloat16()
    q, lse = torch.randn(6, 4, 64, device="cuda").bfloat16(), torch.full((6, 4), 3.0, device="cuda")
    a = sv.make_weigh_args(q=q, lse=lse, cu_rows=i32([0, 4, 6]), max_rows=4, cache=sv.make_cache(k, k),
                           block_table=i32([[0, 3, 5, 2, 1], [7, 6, 4, 0, 0]]), kv_len=i32(lens))
    want = {ld: sv.spec_attention_weights(a, ld=ld)[0].clone() for ld in (70, 129)}
    got = {}
    torch.cuda.synchronize()

    def work(ld):
        stream = torch.cuda.Stream()
        outs = [torch.full((2, 2, ld), -1.0, device="cuda") for _ in range(200)]
        torch.cuda.synchronize()
        for o in outs:
            sv.spec_attention_weights(a, out=o, stream=stream)
        stream.synchronize()
        got[ld] = outs

    threads = [threading.Thread(target=work, args=(ld,)) for ld in want]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for ld, w in want.items():
        assert all(torch.equal(o, w) for o in got[ld])
