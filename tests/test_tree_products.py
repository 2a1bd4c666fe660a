"""Sizes whose product passes 64 bits are refused as those that pass 32 bits
are: 2^64 is not 0."""
import ctypes

import pytest

import speculative_decoding_verification_23_gb300 as sv
import test_tree_abi as abi
from test_tree_abi import lib  # noqa: F401 (a fixture)

PTR = abi.PTR


@pytest.mark.parametrize("B,heads,keep", [(1 << 30, 1 << 30, 1 << 7), (1 << 30, 1 << 29, 1 << 8), (1 << 16, 1 << 16, 8),
                                          (1 << 30, 1, 16)])
def test_eviction(lib, B, heads, keep):
    a = abi.evict_args(B=B, cache_heads=heads, keep=keep, ld_to=1 << 10)
    assert lib.spec_cache_evict(ctypes.byref(a), PTR, None, PTR, None, None) == sv.SPEC_ERR_SHAPE


@pytest.mark.parametrize("ld_path,heads,dim", [(1 << 30, 1 << 30, 128), (1 << 30, 1 << 29, 256), (1 << 20, 1 << 10, 64)])
def test_paths(lib, ld_path, heads, dim):
    a = abi.commit_args(ld_path=ld_path, cache_heads=heads, cache_dim=dim)
    assert lib.spec_cache_commit(ctypes.byref(a), PTR, None, None) == sv.SPEC_ERR_SHAPE


@pytest.mark.parametrize("B,keep,outer,row_bytes", [
    (1 << 16, 1 << 16, 1 << 16, 1 << 30),             # 2^64 blocks of 16 KB
    (1 << 16, 1 << 16, (1 << 31) - 1, 1 << 40),
    (1 << 30, 1 << 30, 1, 16), (1 << 20, 1 << 10, 2, 16),
])
def test_states(lib, B, keep, outer, row_bytes):
    s = sv.SpecBeamState()
    s.src = s.dst = PTR
    s.row_bytes, s.outer = row_bytes, outer
    assert lib.spec_beam_reorder(B, 4, keep, PTR, ctypes.byref(s), 1, None) == sv.SPEC_ERR_SHAPE


def test_many_states(lib):
    """Eight states of 2^61 blocks less some: their sum is below 0 in 64 bits."""
    s = sv.SpecBeamState()
    s.src = s.dst = PTR + 1
    s.row_bytes, s.outer = 1 << 40, 1
    block = (sv.SpecBeamState * 8)(*[s] * 8)
    assert lib.spec_beam_reorder((1 << 31) - 1, 4, 1, PTR, block, 8, None) == sv.SPEC_ERR_SHAPE
