"""Sizes at the edge of 32-bit positions are refused before any launch."""
import ctypes

import pytest

import speculative_decoding_verification_23_gb300 as sv
import test_tree_abi as abi
from test_tree_abi import lib  # noqa: F401 (a fixture)

TOP = 2 ** 31 - 1
PTR = abi.PTR


def calls(lib):
    ref = ctypes.byref
    return [
        (abi.tree_args, lambda a: lib.spec_tree_attention(ref(a), PTR, 256, 64, None, None, PTR, 1 << 40, None)),
        (abi.weigh_args, lambda a: lib.spec_attention_weights(ref(a), None, PTR, None, None)),
        (abi.evict_args, lambda a: lib.spec_cache_evict(ref(a), PTR, None, PTR, None, None)),
        (abi.commit_args, lambda a: lib.spec_cache_commit(ref(a), PTR, None, None)),
    ]


@pytest.mark.parametrize("which", range(4))
def test_tables_end_before_the_last_32_bit_position(lib, which):
    make, call = calls(lib)[which]
    assert call(make(cache_page_size=1, ld_table=TOP)) == sv.SPEC_ERR_SHAPE
    assert call(make(cache_page_size=1, ld_table=TOP - 65534)) == sv.SPEC_ERR_SHAPE


@pytest.mark.parametrize("which", [1, 2])
def test_rows_of_weights_end_before_the_last_32_bit_position(lib, which):
    make, call = calls(lib)[which]
    assert call(make(ld=TOP)) == sv.SPEC_ERR_SHAPE
    assert call(make(ld=TOP - 65534)) == sv.SPEC_ERR_SHAPE


def test_paths_end_before_the_last_32_bit_piece(lib):
    make, call = calls(lib)[3]
    assert call(make(ld_path=TOP // 16)) == sv.SPEC_ERR_SHAPE
