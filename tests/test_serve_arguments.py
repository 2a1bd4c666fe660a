"""What the binding of the operators beside the drafted tree refuses before it calls the library."""
import pytest

import speculative_decoding_verification_23_gb300 as sv
from speculative_decoding_verification_23_gb300 import serve
from test_tree_arguments import Fake, f32, i32, kv

torch = pytest.importorskip("torch")


def e4m3(*shape):
    return Fake(torch.zeros(shape, dtype=torch.float8_e4m3fn))


def cache8():
    return sv.make_cache8(e4m3(4, 16, 2, 64), e4m3(4, 16, 2, 64), f32(4, 2, 2), f32(4, 2, 2))


def drafted(cache, **kw):
    a = dict(q=kv(3, 4, 64), k_new=kv(3, 2, 64), v_new=kv(3, 2, 64), cu_nodes=i32(3), max_nodes=2, ctx_len=i32(2),
             cache=cache, block_table=i32(2, 2), tree_mask=i32(3, 1))
    a.update(kw)
    return a


def rotate(**kw):
    a = dict(q=kv(3, 4, 64), k=kv(3, 2, 64), positions=i32(3), inv_freq=f32(32), q_weight=kv(64), k_weight=kv(64))
    a.update(kw)
    return a


def commit(**kw):
    a = dict(k_new=kv(1, 3, 2, 64), v_new=kv(1, 3, 2, 64), cu_nodes=i32(3), path=i32(2, 2), path_len=i32(2), cache=cache8(),
             block_table=i32(2, 2), ctx_len=i32(2))
    a.update(kw)
    return a


def window(**kw):
    return dict(drafted(sv.make_cache(kv(4, 16, 2, 64), kv(4, 16, 2, 64)), **kw), **{"window": 8, "sinks": 1, **kw})


def test_what_is_right_is_taken():
    a = sv.make_rotate_args(**rotate())
    assert (a.rows, a.heads_q, a.heads_k, a.dim, a.rot) == (3, 4, 2, 64, 64)
    assert sv.make_rotate_args(**rotate(q=None, q_weight=None)).heads_q == 0
    a = sv.make_window_args(**window())
    assert (a.tree.B, a.tree.total_nodes, a.window, a.sinks) == (2, 3, 8, 1)
    a = sv.make_cache8_args(**drafted(cache8(), window=8, sinks=1))
    assert (a.B, a.mask_words, a.cache.block, a.window, a.sinks, a.scale) == (2, 1, 8, 8, 1, 0.125)
    a = sv.make_cache8_commit_args(**commit())
    assert (a.B, a.total_nodes, a.ld_path, a.cache.layers) == (2, 3, 2, 1)


@pytest.mark.parametrize("kw", [
    dict(q=None, k=None), dict(q=f32(3, 4, 64)), dict(k=kv(4, 2, 64)), dict(k=kv(3, 2, 128)), dict(positions=f32(3)),
    dict(positions=i32(4)), dict(inv_freq=kv(32)), dict(inv_freq=f32(2, 16)), dict(q_weight=kv(32)), dict(k_weight=f32(64)),
    dict(q=Fake(torch.zeros(3, 64, 4, dtype=torch.bfloat16).transpose(1, 2))), dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16))])
def test_rotation(kw):
    with pytest.raises((TypeError, ValueError)):
        sv.make_rotate_args(**rotate(**kw))


@pytest.mark.parametrize("kw", [dict(window=None), dict(sinks=-1 << 32), dict(window=1 << 31), dict(max_nodes=2 + (1 << 32))])
def test_windows(kw):
    with pytest.raises((TypeError, ValueError)):
        sv.make_window_args(**window(**kw))


@pytest.mark.parametrize("shapes", [
    [(4, 16, 2), (4, 16, 2), (4, 2), (4, 2)], [(4, 16, 2, 64), (4, 16, 2, 32), (4, 2, 2), (4, 2, 2)],
    [(4, 16, 2, 64), (4, 16, 2, 64), (4, 2, 2), (4, 1, 2)], [(4, 16, 2, 64), (4, 16, 2, 64), (4, 3, 2), (4, 3, 2)],
    [(4, 16, 2, 64), (4, 16, 2, 64), (3, 2, 2), (3, 2, 2)], [(4, 16, 2, 64), (4, 16, 2, 64), (4, 2, 1), (4, 2, 1)],
    [(2, 4, 16, 2, 64), (2, 4, 16, 2, 64), (4, 2, 2), (4, 2, 2)], [(4, 16, 2, 64), (4, 16, 2, 64), (4, 0, 2), (4, 0, 2)]])
def test_shapes_of_a_cache(shapes):
    with pytest.raises((TypeError, ValueError)):
        sv.make_cache8(*(e4m3(*s) for s in shapes[:2]), *(f32(*s) for s in shapes[2:]))


def test_types_and_strides_of_a_cache():
    good = [e4m3(4, 16, 2, 64), e4m3(4, 16, 2, 64), f32(4, 2, 2), f32(4, 2, 2)]
    for i, other in ((0, kv(4, 16, 2, 64)), (1, Fake(torch.zeros(4, 16, 2, 64, dtype=torch.uint8))), (2, kv(4, 2, 2)),
                     (3, torch.zeros(4, 2, 2)), (1, Fake(torch.zeros(4, 2, 16, 64, dtype=torch.float8_e4m3fn).transpose(1, 2))),
                     (3, Fake(torch.zeros(4, 2, 2).transpose(1, 2)))):
        with pytest.raises((TypeError, ValueError)):
            sv.make_cache8(*good[:i], other, *good[i + 1:])


@pytest.mark.parametrize("kw", [
    dict(q=kv(3, 4, 128)), dict(k_new=kv(3, 4, 64)), dict(v_new=kv(4, 2, 64)), dict(q=f32(3, 4, 64)), dict(cu_nodes=f32(3)),
    dict(v_new=Fake(torch.zeros(2, 3, 64, dtype=torch.bfloat16).transpose(0, 1))), dict(ctx_len=i32(3)),
    dict(block_table=i32(3, 2)), dict(tree_mask=i32(2, 1)), dict(tree_mask=f32(3, 1)), dict(layer=1 << 32), dict(window=1 << 31),
    dict(sinks=None), dict(max_nodes=None)])
def test_attention_over_8_bits(kw):
    with pytest.raises((TypeError, ValueError)):
        sv.make_cache8_args(**drafted(cache8(), **kw))


@pytest.mark.parametrize("kw", [
    dict(k_new=kv(1, 3, 4, 64)), dict(v_new=kv(1, 4, 2, 64)), dict(k_new=f32(1, 3, 2, 64)), dict(k_new=kv(2, 3, 2, 64), v_new=kv(2, 3, 2, 64)),
    dict(path=i32(3, 2)), dict(path=f32(2, 2)), dict(path_len=i32(3)), dict(ctx_len=i32(1)), dict(block_table=i32(1, 2))])
def test_commitment_to_8_bits(kw):
    with pytest.raises((TypeError, ValueError)):
        sv.make_cache8_commit_args(**commit(**kw))


def test_results(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    monkeypatch.setattr(serve, "_lib", Lib)
    a = sv.make_rotate_args(**rotate())
    for kw in (dict(out_q=kv(3, 2, 64)), dict(out_q=f32(3, 4, 64)), dict(out_q=torch.zeros(3, 4, 64, dtype=torch.bfloat16))):
        with pytest.raises((TypeError, ValueError)):
            sv.spec_norm_rotate(a, out_k=kv(3, 2, 64), **kw)
    c = sv.make_cache8_commit_args(**commit())
    for kw in (dict(out_len=i32(3)), dict(out_len=f32(2)), dict(out_len=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises((TypeError, ValueError)):
            sv.spec_cache8_commit(c, **kw)
