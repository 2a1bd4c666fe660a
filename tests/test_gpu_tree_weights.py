"""Attention weights of rows and keys that are not finite."""
import numpy as np
import pytest

import speculative_decoding_verification_23_gb300 as sv
import tree_ref as R
from test_gpu_tree import TYPES, fill, i32, make_kv, make_pages

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def weigh(dim, rows, n, lse_of, k_of=None, dtype="bf16", h=2, hq=6, page=16):
    rng = np.random.default_rng(dim + rows)
    table, num = make_pages(rng, [n], page)
    k, _ = make_kv(rng, num, page, h, dim, dtype, "heads")
    k64 = fill(k, rng, table, [n], page)
    if k_of is not None:
        j, value = k_of
        k[int(table[0, j // page]), j % page, :, 0] = value
    q = torch.from_numpy(rng.standard_normal((rows, hq, dim)).astype(np.float32)).to("cuda", TYPES[dtype])
    q[:, :, 0] = 1.0
    lse = torch.from_numpy(rng.uniform(1, 6, (rows, hq)).astype(np.float32)).cuda()
    for at, value in lse_of.items():
        lse[at] = value
    a = sv.make_weigh_args(q=q, lse=lse, cu_rows=i32([0, rows]), max_rows=rows, cache=sv.make_cache(k, k),
                           block_table=i32(table), kv_len=i32([n]))
    out, st = sv.spec_attention_weights(a, ld=n)
    assert st.tolist() == [0]
    return R.f64(out), R.f64(q), lse, k64, table


# both kernels: 64 and 128 channels on tensor memory, 96 on warps
DIMS = [64, 96, 128]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_rows_of_infinite_lse_add_nothing(dim, value):
    rows, n = 5, 300
    out, q, lse, k64, table = weigh(dim, rows, n, {(1, 0): value, (4, 3): value})
    finite = lse.clone()
    finite[torch.isinf(lse)] = float("inf")
    want, tol = R.weights(q, R.f64(finite), [0, rows], k64, 16, table, [n], dim ** -0.5, None, n)
    assert np.all(np.abs(out - want) <= tol)


@pytest.mark.parametrize("dim", DIMS)
def test_a_row_of_no_number_reaches_the_keys_it_sees(dim):
    rows, n = 5, 300
    out = weigh(dim, rows, n, {(1, 0): float("nan")})[0]
    # row 1 sees keys up to n - rows + 1; query head 0 belongs to key head 0
    assert np.all(np.isnan(out[0, 0, :n - rows + 2])) and np.all(np.isfinite(out[0, 0, n - rows + 2:]))
    assert np.all(np.isfinite(out[0, 1]))


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("rows", [1, 5, 11])  # 3, 15 and 33 rows per key head: all but whole tiles
def test_a_key_of_minus_infinity_has_weight_zero(dim, rows):
    n, j = 300, 40
    out = weigh(dim, rows, n, {}, (j, -float("inf")))[0]
    assert np.all(out[0, :, j] == 0)
    others = np.delete(out[0], j, axis=1)
    assert np.all(np.isfinite(others)) and np.all(others > 0)
