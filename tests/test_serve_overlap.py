"""Results that overlap what they must not: refused on the host, before anything runs."""
import ctypes

import pytest

import speculative_decoding_verification_23_gb300 as sv
from test_serve_abi import PTR, _gpu, cache8_args, commit8_args, lib, rotate, rotate_args  # noqa: F401

# where a call that is not refused ends: at the missing device (with one it would run, on addresses that are none)
pytestmark = pytest.mark.skipif(_gpu(), reason="the calls that are right would run")
TAKEN = sv.SPEC_ERR_DEVICE


@pytest.mark.parametrize("oq,code", [
    ((256, 64), TAKEN), ((64, 256), TAKEN), ((1024, 128), TAKEN), ((0, 64), sv.SPEC_ERR_SHAPE), ((256, 0), sv.SPEC_ERR_SHAPE),
    ((0, 0), sv.SPEC_ERR_SHAPE), ((256, 56), sv.SPEC_ERR_SHAPE), ((248, 64), sv.SPEC_ERR_SHAPE), ((64, 248), sv.SPEC_ERR_SHAPE),
    ((64, 64), sv.SPEC_ERR_SHAPE), ((56, 256), sv.SPEC_ERR_SHAPE)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_and_heads_of_a_result_overlap(lib, oq, code, in_place):  # noqa: F811
    """4 rows of 4 heads of 64 channels.  In place of rows that share memory too."""
    a = rotate_args(q=7 * PTR, sq_row=oq[0], sq_head=oq[1]) if in_place else rotate_args()
    assert rotate(lib, a, out_q=7 * PTR, oq=oq) == code
    b = rotate_args(heads_q=2, heads_k=4, sk_row=oq[0], sk_head=oq[1], k=7 * PTR) if in_place else rotate_args(heads_q=2, heads_k=4)
    assert rotate(lib, b, out_k=7 * PTR, ok=oq) == code


def test_strides_of_a_single_row_or_head_are_free(lib):  # noqa: F811
    assert rotate(lib, rotate_args(rows=1), oq=(0, 64), ok=(0, 64)) == TAKEN
    assert rotate(lib, rotate_args(heads_q=1, heads_k=1), oq=(64, 0), ok=(64, 0)) == TAKEN
    assert rotate(lib, rotate_args(rows=1), oq=(0, 56)) == sv.SPEC_ERR_SHAPE
    assert rotate(lib, rotate_args(heads_k=0, k=None), out_k=None, ok=(0, 0)) == TAKEN
    # inputs may be one row many times over
    assert rotate(lib, rotate_args(sq_row=0, sk_row=0, sk_head=0)) == TAKEN


# the scales of 8 pages, 2 blocks, 2 heads: 32 of 4 bytes
@pytest.mark.parametrize("at", [3 * PTR, 3 * PTR + 124, 4 * PTR - 4, 4 * PTR + 64])
def test_attention_results_over_the_scales(lib, at):  # noqa: F811
    a = cache8_args()
    n = lib.spec_cache8_workspace_bytes(ctypes.byref(a))

    def call(lse, status, a=a):
        return lib.spec_cache8_attention(ctypes.byref(a), 9 * PTR, 256, 64, lse, status, 16 * PTR, 1 << 30, None)

    assert n > 0 and call(10 * PTR, 11 * PTR) == TAKEN
    # without a device the checks of overlaps come after the sizes'
    assert call(at, 11 * PTR) == sv.SPEC_ERR_SHAPE and call(10 * PTR, at) == sv.SPEC_ERR_SHAPE
    assert call(3 * PTR + 128, 4 * PTR + 128) == TAKEN


@pytest.mark.parametrize("at", [3 * PTR, 3 * PTR + 124, 4 * PTR - 4, 4 * PTR + 64])
def test_commitment_results_over_the_scales(lib, at):  # noqa: F811
    a = commit8_args()

    def call(length, status):
        return lib.spec_cache8_commit(ctypes.byref(a), length, status, None)

    assert call(10 * PTR, 11 * PTR) == TAKEN and call(3 * PTR + 128, 4 * PTR + 128) == TAKEN
    assert call(at, 11 * PTR) == sv.SPEC_ERR_SHAPE and call(10 * PTR, at) == sv.SPEC_ERR_SHAPE
