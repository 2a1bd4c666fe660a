"""The measured cases' plain forms of commitment and eviction move rows, so
they equal the definition bit by bit, whatever the lengths."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("operator_cases", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.DEV = "cpu"
    return m


def same(ops, case, seed):
    got, want = ops.run(ops.prepare(case, seed)), ops.exact(case, seed)
    assert got.keys() == want.keys()
    for name in got:
        assert torch.equal(torch.as_tensor(got[name]).double(), torch.as_tensor(want[name]).double()), name


@pytest.mark.parametrize("batch,nodes,lo,hi,page", [(7, 33, 10, 100, 16), (1, 9, 77, 77, 16), (12, 64, 1, 40, 32),
                                                    (5, 1, 3, 200, 8), (9, 20, 100, 101, 64)])
@pytest.mark.parametrize("ragged", [False, True])
def test_commitment(ops, batch, nodes, lo, hi, page, ragged):
    for seed in range(8):
        same(ops, dict(op="commit", layers=2, batch=batch, nodes=nodes, ragged=ragged, kv_heads=1, dim=64, ctx_lo=lo,
                       ctx_hi=hi, page=page, dtype="bf16"), seed)


@pytest.mark.parametrize("batch,lo,hi,keep,sink,recent,page", [(6, 20, 300, 100, 4, 30, 16), (1, 90, 90, 17, 0, 0, 16),
                                                               (9, 5, 64, 33, 0, 16, 8), (4, 10, 500, 250, 4, 0, 128)])
def test_eviction(ops, batch, lo, hi, keep, sink, recent, page):
    for seed in range(4):
        same(ops, dict(op="evict", batch=batch, kv_heads=2, dim=64, len_lo=lo, len_hi=hi, keep=keep, sink=sink,
                       recent=recent, page=page, dtype="fp16"), seed)
