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


class Fake:
    """A CPU tensor that passes for a CUDA one: no memory is touched."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def i32(*shape):
    return Fake(torch.zeros(shape, dtype=torch.int32))


def f32(*shape):
    return Fake(torch.zeros(shape))


def kv(*shape):
    return Fake(torch.zeros(shape, dtype=torch.bfloat16))


def makers():
    cache = sv.make_cache(kv(4, 16, 2, 64), kv(4, 16, 2, 64))
    both = dict(cache=cache, block_table=i32(2, 2))
    tree_args = dict(q=kv(3, 4, 64), k_new=kv(3, 2, 64), v_new=kv(3, 2, 64), cu_nodes=i32(3), max_nodes=2, layer=0,
                     ctx_len=i32(2), **both)
    weigh = dict(q=kv(3, 4, 64), lse=f32(3, 4), cu_rows=i32(3), max_rows=2, layer=0, kv_len=i32(2), **both)
    evict = dict(weights=f32(2, 2, 30), kv_len=i32(2), keep=8, sink=1, recent=2, layer=0, to_table=i32(2, 1), **both)
    beams = dict(logits=f32(6, 12), V=10, scores=f32(2, 3), keep=2, finished=i32(2, 3), end_token=3)
    return [(sv.make_tree_args, tree_args, ("max_nodes", "layer")), (sv.make_weigh_args, weigh, ("max_rows", "layer")),
            (sv.make_evict_args, evict, ("keep", "sink", "recent", "layer")),
            (sv.make_beam_args, beams, ("keep", "end_token"))]


@pytest.mark.parametrize("which", range(4))
def test_whole_numbers_fit_their_fields(which):
    make, kw, names = makers()[which]
    a = make(**kw)
    for name in names:
        assert getattr(a, name) == kw[name]
        for more in (1 << 32, -1 << 32, 1 << 31):
            with pytest.raises(ValueError, match=name):
                make(**{**kw, name: kw[name] + more})


def test_the_beams_fit_their_field(no_library):
    with pytest.raises(ValueError, match="beams"):
        sv.make_reorder_args(parents=i32(2, 2), beams=3 + (1 << 32), states=[])


def test_the_row_length_fits_its_field(monkeypatch):
    monkeypatch.setattr(tree, "_lib", lambda: None)
    with pytest.raises(ValueError, match="ld"):
        sv.spec_attention_weights(sv.SpecWeighArgs(), ld=1 << 32)
