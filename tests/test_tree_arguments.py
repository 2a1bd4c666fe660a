"""What the binding refuses before it calls the library."""
import pytest

import speculative_decoding_verification_23_gb300 as sv
from speculative_decoding_verification_23_gb300 import tree

torch = pytest.importorskip("torch")


@pytest.fixture
def no_library(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    monkeypatch.setattr(tree, "_lib", Lib)


@pytest.mark.parametrize("workspace", [torch.empty(1 << 16, dtype=torch.uint8), torch.empty(64, 64).t()[1:]])
def test_a_workspace_is_on_the_device(no_library, workspace):
    a = sv.SpecTreeArgs()
    a.B, a.total_nodes, a.heads_q, a.cache.dim, a.torch_dtype = 1, 1, 1, 64, torch.bfloat16
    with pytest.raises(TypeError, match="workspace"):
        sv.spec_tree_attention(a, workspace=workspace)
    b = sv.SpecBeamArgs()
    b.B = b.W = b.keep = b.V = 1
    with pytest.raises(TypeError, match="workspace"):
        sv.spec_beam_select(b, workspace=workspace)


def test_a_workspace_counts_in_bytes():
    class OnDevice:
        is_cuda = True

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

    assert tree._workspace_bytes(OnDevice(torch.empty(100, dtype=torch.float32))) == 400
    assert tree._workspace_bytes(OnDevice(torch.empty(100, dtype=torch.uint8))) == 100
    with pytest.raises(TypeError):
        tree._workspace_bytes(OnDevice(torch.empty(8, 8)[:, ::2]))
