"""Pages outside the cache: what of a request they spoil, and what is said."""
import numpy as np
import pytest

import speculative_decoding_verification_23_gb300 as sv
import tree_ref as R
from test_gpu_tree import TYPES, fill, i32, make_kv, make_pages

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dim,page,rows", [
    (64, 16, 4), (128, 64, 4),                        # tensor memory
    (96, 1, 4), (96, 3, 4), (96, 8, 4), (96, 24, 4), (192, 5, 4), (256, 16, 4),
    (64, 3, 4), (64, 12, 4), (64, 8, 140),            # other pages, and more rows: warps
])
def test_weights_of_a_bad_page_alone_are_spoiled(dim, page, rows):
    rng = np.random.default_rng(dim + page)
    lens, n = [211, 190], [rows, 3]
    table, num = make_pages(rng, lens, page)
    k, _ = make_kv(rng, num, page, 2, dim, "bf16", "heads")
    k64 = fill(k, rng, table, lens, page)
    cu = np.concatenate([[0], np.cumsum(n)])
    q = torch.from_numpy(rng.standard_normal((cu[-1], 4, dim)).astype(np.float32)).to("cuda", TYPES["bf16"])
    lse = torch.from_numpy(rng.uniform(1, 6, (cu[-1], 4)).astype(np.float32)).cuda()
    before = torch.from_numpy(rng.uniform(0, 9, (2, 2, 220)).astype(np.float32)).cuda()
    want, tol = R.weights(R.f64(q), R.f64(lse), cu, k64, page, table, lens, dim ** -0.5, R.f64(before), 220)
    bad = {0, 2, (lens[0] - 1) // page}
    for p, to in zip(sorted(bad), (num, -1, 1 << 30)):
        table[0, p] = to
    a = sv.make_weigh_args(q=q, lse=lse, cu_rows=i32(cu), max_rows=max(n), cache=sv.make_cache(k, k),
                           block_table=i32(table), kv_len=i32(lens))
    out, st = sv.spec_attention_weights(a, before)
    assert st.tolist() == [sv.SPEC_STATUS_BAD_PAGE, 0]
    got = R.f64(out)
    j = np.arange(220)
    spoiled = np.isin(j // page, list(bad)) & (j < lens[0])
    assert np.all(np.isnan(got[0][:, spoiled])) and np.all(np.isfinite(got[0][:, ~spoiled]))
    got[0][:, spoiled] = want[0][:, spoiled]
    assert np.all(np.abs(got - want) <= tol)
