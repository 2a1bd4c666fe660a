"""Attention weights where some requests, or all, bring no rows: many more
tiles than CTAs, so that a CTA passes over several such requests."""
import numpy as np
import pytest

import speculative_decoding_verification_23_gb300 as sv
import tree_ref as R
from test_gpu_tree import TYPES, fill, i32, make_kv, make_pages

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def rows_of(kind, n, lens):
    """Rows of each request."""
    few = [min(x, 1 + i % 4) for i, x in enumerate(lens)]
    idle = {"none": lambda i: False, "odd": lambda i: i % 2 == 1, "runs": lambda i: (i // 5) % 3 != 0,
            "all": lambda i: True, "all but the last": lambda i: i < n - 1}[kind]
    return [0 if idle(i) else few[i] for i in range(n)]


def call(seed, lens, rows, hq, h, dim, page, dtype, with_before, break_at=()):
    rng = np.random.default_rng(seed)
    table, num = make_pages(rng, lens, page)
    k, _ = make_kv(rng, num, page, h, dim, dtype, "heads")
    k64 = fill(k, rng, table, lens, page)
    cu = np.concatenate([[0], np.cumsum(rows)])
    q = torch.from_numpy((2 * rng.standard_normal((cu[-1], hq, dim))).astype(np.float32)).to("cuda", TYPES[dtype])
    lse = torch.from_numpy(rng.uniform(1, 6, (cu[-1], hq)).astype(np.float32)).cuda()
    ld = max(lens) + 5
    before = torch.from_numpy(rng.uniform(0, 9, (len(rows), h, ld)).astype(np.float32)).cuda() if with_before else None
    want, tol = R.weights(R.f64(q), R.f64(lse), cu, k64, page, table, lens, dim ** -0.5,
                          None if before is None else R.f64(before), ld)
    for b, p in break_at:
        table[b, p] = num
    a = sv.make_weigh_args(q=q, lse=lse, cu_rows=i32(cu), max_rows=max(1, max(rows)), cache=sv.make_cache(k, k),
                           block_table=i32(table), kv_len=i32(lens))
    return a, before, ld, want, tol


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("with_before", [False, True])
@pytest.mark.parametrize("kind", ["none", "odd", "runs", "all", "all but the last"])
def test_requests_without_rows_keep_their_weights(kind, with_before, dim):
    n = 128
    lens = [1 + (37 * i) % 100 if i % 16 else 300 for i in range(n)]
    rows = rows_of(kind, n, lens)
    a, before, ld, want, tol = call(dim, lens, rows, 16, 8, dim, 16, "bf16", with_before)
    out, st = sv.spec_attention_weights(a, before, ld=ld)
    assert st.tolist() == [0] * n
    assert np.all(np.abs(R.f64(out) - want) <= tol)
    for b in range(n):
        if rows[b] == 0 and with_before:
            assert torch.equal(out[b, :, :lens[b]], before[b, :, :lens[b]])
    if with_before:  # in place
        sv.spec_attention_weights(a, before, out=before)
        assert torch.equal(before, out)


@pytest.mark.parametrize("page", [16, 64])
def test_a_long_cache_without_rows(page):
    lens, rows = [9001, 40, 20003, 700], [0, 3, 0, 0]
    a, before, ld, want, tol = call(5, lens, rows, 14, 2, 64, page, "fp16", True, break_at=[(2, 3)])
    out, st = sv.spec_attention_weights(a, before, ld=ld)
    assert st.tolist() == [0, 0, sv.SPEC_STATUS_BAD_PAGE, 0]
    bad = np.zeros(ld, bool)
    bad[3 * page:4 * page] = True
    got = R.f64(out)
    assert np.all(np.isnan(got[2][:, bad])) and np.all(np.isfinite(got[2][:, ~bad]))
    got[2][:, bad] = want[2][:, bad]
    assert np.all(np.abs(got - want) <= tol)
