"""The C ABI of the operators beside the drafted tree, and its refusals: nothing here computes on a GPU."""
import ctypes
import os
import re
import subprocess

import pytest

import speculative_decoding_verification_23_gb300 as sv
from speculative_decoding_verification_23_gb300 import serve

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"spec_rotate_args": sv.SpecRotateArgs, "spec_window_args": sv.SpecWindowArgs, "spec_cache8": sv.SpecCache8,
           "spec_cache8_args": sv.SpecCache8Args, "spec_cache8_commit_args": sv.SpecCache8CommitArgs}
PTR = 1 << 20  # never followed: every call below is refused


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return serve._lib()


def test_header_and_library_declare_the_python_names(lib):
    text = open(os.path.join(ROOT, "include", "spec_serve.h")).read()
    names = sorted(set(re.findall(r"^(?:size_t|int) (spec_\w+)\(", text, re.M)))
    assert names == sorted(sv.EXPORTED_SERVE)
    out = subprocess.run(["nm", "-D", "--defined-only", sv.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r" T (spec_\w+)", out))


@pytest.mark.parametrize("name", sorted(STRUCTS))
def test_struct_layout_matches_header(tmp_path, name):
    cls = STRUCTS[name]
    body = "\n".join(f'  printf("{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spec_serve.h"\nint main(void) {\n' + body +
                   f'\n  printf("size %zu\\n", sizeof({name}));\n  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for f in cls._fields_:
        assert int(got[f[0]]) == getattr(cls, f[0]).offset, f[0]
    assert int(got["size"]) == ctypes.sizeof(cls)


def _set(x, kw):
    for k, v in kw.items():
        obj, name = x, k
        if k.startswith("cache_"):
            obj, name = (x.tree.cache if hasattr(x, "tree") else x.cache), k[6:]
        elif k.startswith("tree_") and hasattr(x, "tree"):
            obj, name = x.tree, k[5:]
        assert name in [f[0] for f in obj._fields_], k
        setattr(obj, name, v)
    return x


# ------------------------------------------------------------------ rotation

def rotate_args(**kw):
    a = sv.SpecRotateArgs()
    a.rows, a.heads_q, a.heads_k, a.dim, a.rot, a.dtype, a.eps = 4, 4, 2, 64, 64, sv.SPEC_BF16, 1e-6
    a.q, a.k, a.positions, a.inv_freq = PTR, 2 * PTR, 3 * PTR, 4 * PTR
    a.sq_row, a.sq_head, a.sk_row, a.sk_head = 256, 64, 128, 64
    return _set(a, kw)


def rotate(lib, a, out_q=5 * PTR, oq=(256, 64), out_k=6 * PTR, ok=(128, 64)):
    return lib.spec_norm_rotate(None if a is None else ctypes.byref(a), out_q, *oq, out_k, *ok, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=sv.SPEC_F32), sv.SPEC_ERR_DTYPE), (dict(rows=-1), sv.SPEC_ERR_SHAPE), (dict(heads_q=-1), sv.SPEC_ERR_SHAPE),
    (dict(heads_k=70000), sv.SPEC_ERR_SHAPE), (dict(dim=80), sv.SPEC_ERR_SHAPE), (dict(rot=4), sv.SPEC_ERR_SHAPE),
    (dict(rot=72), sv.SPEC_ERR_SHAPE), (dict(rot=-8), sv.SPEC_ERR_SHAPE), (dict(eps=-1.0), sv.SPEC_ERR_SHAPE),
    (dict(eps=float("nan")), sv.SPEC_ERR_SHAPE), (dict(q=None), sv.SPEC_ERR_NULL), (dict(k=None), sv.SPEC_ERR_NULL),
    (dict(positions=None), sv.SPEC_ERR_NULL), (dict(inv_freq=None), sv.SPEC_ERR_NULL), (dict(q=PTR + 8), sv.SPEC_ERR_ALIGN),
    (dict(sk_head=60), sv.SPEC_ERR_ALIGN), (dict(sq_row=-256), sv.SPEC_ERR_ALIGN), (dict(q_weight=PTR + 2), sv.SPEC_ERR_ALIGN),
    (dict(q_weight=5 * PTR), sv.SPEC_ERR_SHAPE), (dict(positions=6 * PTR + 16), sv.SPEC_ERR_SHAPE),
])
def test_rotation_refuses(lib, kw, code):
    assert rotate(lib, rotate_args(**kw)) == code


def test_rotation_refuses_its_buffers(lib):
    a = rotate_args()
    assert rotate(lib, None) == sv.SPEC_ERR_NULL
    assert rotate(lib, a, out_q=None) == sv.SPEC_ERR_NULL
    assert rotate(lib, a, out_k=6 * PTR + 4) == sv.SPEC_ERR_ALIGN
    assert rotate(lib, a, oq=(252, 64)) == sv.SPEC_ERR_ALIGN
    assert rotate(lib, a, out_q=PTR + 128) == sv.SPEC_ERR_SHAPE             # half over its input
    assert rotate(lib, a, out_q=PTR, oq=(512, 64)) == sv.SPEC_ERR_SHAPE     # in place, other strides
    assert rotate(lib, a, out_q=2 * PTR) == sv.SPEC_ERR_SHAPE               # over the keys
    assert rotate(lib, a, out_k=5 * PTR) == sv.SPEC_ERR_SHAPE               # both results at one place


def test_parts_of_one_projection_are_told_apart(lib):
    """Queries, keys and values side by side in rows of 512: in place is allowed (and ends at the missing device), a
    result over another's columns is not."""
    a = rotate_args(q=PTR, k=PTR + 512, sq_row=512, sk_row=512)
    ok = {sv.SPEC_ERR_DEVICE} if not _gpu() else None
    if ok:
        assert rotate(lib, a, out_q=PTR, oq=(512, 64), out_k=PTR + 512, ok=(512, 64)) in ok
        assert rotate(lib, a, out_q=PTR + 768, oq=(512, 64), out_k=PTR + 512, ok=(512, 64)) == sv.SPEC_ERR_SHAPE
    assert rotate(lib, a, out_q=PTR + 256, oq=(512, 64), out_k=6 * PTR) == sv.SPEC_ERR_SHAPE
    assert rotate(lib, a, out_q=5 * PTR, out_k=PTR + 384, ok=(512, 64)) == sv.SPEC_ERR_SHAPE


def _gpu():
    import torch

    return torch.cuda.is_available()


# -------------------------------------------------------------------- window

def window_args(**kw):
    a = sv.SpecWindowArgs()
    t = a.tree
    t.B, t.total_nodes, t.max_nodes, t.heads_q, t.scale = 2, 6, 4, 4, 0.125
    t.cu_nodes = t.q = t.k_new = t.v_new = t.block_table = t.ctx_len = PTR
    t.sq_node, t.sq_head, t.sn_node, t.sn_head, t.ld_table = 256, 64, 128, 64, 4
    c = t.cache
    c.k = c.v = PTR
    c.dtype, c.layers, c.num_pages, c.page_size, c.heads, c.dim = sv.SPEC_BF16, 1, 8, 16, 2, 64
    c.s_layer, c.s_page, c.s_slot, c.s_head = 0, 2048, 128, 64
    a.window, a.sinks = 32, 4
    return _set(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(window=0), sv.SPEC_ERR_SHAPE), (dict(window=-3), sv.SPEC_ERR_SHAPE), (dict(sinks=-1), sv.SPEC_ERR_SHAPE),
    (dict(cache_k=None), sv.SPEC_ERR_NULL), (dict(cache_dtype=sv.SPEC_F32), sv.SPEC_ERR_DTYPE),
    (dict(cache_dim=80), sv.SPEC_ERR_SHAPE), (dict(cache_s_slot=68), sv.SPEC_ERR_ALIGN),
    (dict(tree_max_nodes=257), sv.SPEC_ERR_SHAPE), (dict(tree_heads_q=3), sv.SPEC_ERR_SHAPE),
    (dict(tree_scale=float("nan")), sv.SPEC_ERR_SHAPE), (dict(tree_q=PTR + 2), sv.SPEC_ERR_ALIGN),
    (dict(tree_tree_mask=PTR, tree_mask_words=0), sv.SPEC_ERR_SHAPE), (dict(tree_ctx_len=None), sv.SPEC_ERR_NULL),
    (dict(tree_B=0), sv.SPEC_ERR_SHAPE), (dict(tree_layer=1), sv.SPEC_ERR_SHAPE),
])
def test_windows_refuse(lib, kw, code):
    a = window_args(**kw)
    assert lib.spec_window_attention(ctypes.byref(a), PTR, 256, 64, None, None, PTR, 1 << 40, None) == code
    assert lib.spec_window_workspace_bytes(ctypes.byref(a)) == 0


# --------------------------------------------------------------- 8-bit cache

def _cache8(c):
    c.k, c.v, c.k_scale, c.v_scale = PTR, 2 * PTR, 3 * PTR, 4 * PTR
    c.layers, c.num_pages, c.page_size, c.heads, c.dim, c.block = 1, 8, 16, 2, 64, 8
    c.s_layer, c.s_page, c.s_slot, c.s_head = 0, 2048, 128, 64
    c.c_layer, c.c_page, c.c_block, c.c_head = 0, 4, 2, 1


def cache8_args(**kw):
    a = sv.SpecCache8Args()
    a.B, a.total_nodes, a.max_nodes, a.heads_q, a.scale, a.dtype = 2, 6, 4, 4, 0.125, sv.SPEC_BF16
    a.cu_nodes = a.q = a.k_new = a.v_new = a.block_table = a.ctx_len = PTR
    a.sq_node, a.sq_head, a.sn_node, a.sn_head, a.ld_table = 256, 64, 128, 64, 4
    _cache8(a.cache)
    return _set(a, kw)


def commit8_args(**kw):
    a = sv.SpecCache8CommitArgs()
    a.B, a.total_nodes, a.dtype, a.ld_path, a.ld_table = 2, 6, sv.SPEC_F16, 4, 4
    a.cu_nodes = a.k_new = a.v_new = a.path = a.path_len = a.block_table = a.ctx_len = PTR
    a.sn_layer, a.sn_node, a.sn_head = 0, 128, 64
    _cache8(a.cache)
    return _set(a, kw)


CACHE8 = [
    (dict(cache_k=None), sv.SPEC_ERR_NULL), (dict(cache_v=None), sv.SPEC_ERR_NULL), (dict(cache_k_scale=None), sv.SPEC_ERR_NULL),
    (dict(cache_v_scale=None), sv.SPEC_ERR_NULL), (dict(cache_layers=0), sv.SPEC_ERR_SHAPE),
    (dict(cache_num_pages=0), sv.SPEC_ERR_SHAPE), (dict(cache_heads=0), sv.SPEC_ERR_SHAPE),
    (dict(cache_dim=32), sv.SPEC_ERR_SHAPE), (dict(cache_block=0), sv.SPEC_ERR_SHAPE), (dict(cache_block=5), sv.SPEC_ERR_SHAPE),
    (dict(cache_block=32), sv.SPEC_ERR_SHAPE), (dict(cache_num_pages=1 << 28), sv.SPEC_ERR_SHAPE),
    (dict(cache_c_page=-1), sv.SPEC_ERR_SHAPE), (dict(cache_k=PTR + 8), sv.SPEC_ERR_ALIGN),
    (dict(cache_v_scale=PTR + 2), sv.SPEC_ERR_ALIGN), (dict(cache_s_slot=136), sv.SPEC_ERR_ALIGN),
    (dict(cache_s_page=-16), sv.SPEC_ERR_ALIGN), (dict(dtype=sv.SPEC_F32), sv.SPEC_ERR_DTYPE),
    (dict(B=0), sv.SPEC_ERR_SHAPE), (dict(total_nodes=-1), sv.SPEC_ERR_SHAPE), (dict(ld_table=0), sv.SPEC_ERR_SHAPE),
    (dict(ld_table=1 << 28), sv.SPEC_ERR_SHAPE), (dict(block_table=None), sv.SPEC_ERR_NULL), (dict(ctx_len=None), sv.SPEC_ERR_NULL),
    (dict(cu_nodes=None), sv.SPEC_ERR_NULL), (dict(k_new=None), sv.SPEC_ERR_NULL), (dict(k_new=PTR + 4), sv.SPEC_ERR_ALIGN),
    (dict(sn_node=60), sv.SPEC_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,code", CACHE8 + [
    (dict(total_nodes=9), sv.SPEC_ERR_SHAPE), (dict(max_nodes=257), sv.SPEC_ERR_SHAPE), (dict(heads_q=3), sv.SPEC_ERR_SHAPE),
    (dict(layer=1), sv.SPEC_ERR_SHAPE), (dict(scale=float("inf")), sv.SPEC_ERR_SHAPE), (dict(window=-1), sv.SPEC_ERR_SHAPE),
    (dict(window=0, sinks=4), sv.SPEC_ERR_SHAPE), (dict(window=4, sinks=-1), sv.SPEC_ERR_SHAPE),
    (dict(q=None), sv.SPEC_ERR_NULL), (dict(sq_head=4), sv.SPEC_ERR_ALIGN), (dict(tree_mask=PTR, mask_words=0), sv.SPEC_ERR_SHAPE),
])
def test_attention_over_8_bits_refuses(lib, kw, code):
    a = cache8_args(**kw)
    assert lib.spec_cache8_attention(ctypes.byref(a), PTR, 256, 64, None, None, PTR, 1 << 40, None) == code
    assert lib.spec_cache8_workspace_bytes(ctypes.byref(a)) == 0


@pytest.mark.parametrize("kind", ["window", "cache8"])
def test_attention_refuses_its_buffers(lib, kind):
    a = window_args() if kind == "window" else cache8_args()
    n = getattr(lib, f"spec_{kind}_workspace_bytes")(ctypes.byref(a))
    assert n > 0

    def call(out=PTR, so=256, ws=PTR, size=n, a=ctypes.byref(a)):
        return getattr(lib, f"spec_{kind}_attention")(a, out, so, 64, None, None, ws, size, None)

    assert call(out=None) == sv.SPEC_ERR_NULL
    assert call(out=PTR + 4) == sv.SPEC_ERR_ALIGN
    assert call(so=257) == sv.SPEC_ERR_ALIGN
    assert call(ws=None) == sv.SPEC_ERR_WORKSPACE
    assert call(ws=PTR + 128) == sv.SPEC_ERR_WORKSPACE
    assert call(size=n - 1) == sv.SPEC_ERR_WORKSPACE
    assert call(a=None) == sv.SPEC_ERR_NULL


@pytest.mark.parametrize("kw,code", CACHE8 + [
    (dict(ld_path=0), sv.SPEC_ERR_SHAPE), (dict(path=None), sv.SPEC_ERR_NULL), (dict(path_len=None), sv.SPEC_ERR_NULL),
    (dict(cache_layers=70000), sv.SPEC_ERR_SHAPE), (dict(ld_path=1 << 30, cache_heads=64), sv.SPEC_ERR_SHAPE),
])
def test_commitment_to_8_bits_refuses(lib, kw, code):
    assert lib.spec_cache8_commit(ctypes.byref(commit8_args(**kw)), 8 * PTR, None, None) == code


def test_commitment_refuses_no_lengths(lib):
    assert lib.spec_cache8_commit(ctypes.byref(commit8_args()), None, None, None) == sv.SPEC_ERR_NULL
    assert lib.spec_cache8_commit(None, 8 * PTR, None, None) == sv.SPEC_ERR_NULL
