"""Argument blocks are read, not written, by the calls that take them."""
import ctypes

import pytest

import speculative_decoding_verification_23_gb300 as sv
from speculative_decoding_verification_23_gb300 import tree

torch = pytest.importorskip("torch")


def test_weights_leave_the_block_as_it_is(monkeypatch):
    """Two threads with one block and rows of different lengths: a call lets
    others run until it is in the library."""
    seen = []

    class Lib:
        @staticmethod
        def spec_attention_weights(args, before, out, status, stream):
            seen.append((args._obj.ld, args._obj.B, args._obj.scale))
            return sv.SPEC_OK

    monkeypatch.setattr(tree, "_lib", lambda: Lib)
    monkeypatch.setattr(tree, "_stream_handle", lambda stream: 0)
    monkeypatch.setattr(tree, "_check_out", lambda *a: None)
    a = sv.SpecWeighArgs()
    a.B, a.scale, a.cache.heads = 2, 0.5, 3
    was = bytes(a)
    status = torch.zeros(2, dtype=torch.int32)
    for ld in (40, 7):
        sv.spec_attention_weights(a, out=torch.zeros(2, 3, ld), out_status=status)
        assert bytes(a) == was
    assert seen == [(40, 2, 0.5), (7, 2, 0.5)]
    assert ctypes.sizeof(a) == len(was)
