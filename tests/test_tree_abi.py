"""The drafted-tree operators' C ABI and its refusals: nothing here computes
on a GPU."""
import ctypes
import os
import re
import subprocess

import pytest

import speculative_decoding_verification_23_gb300 as sv
from speculative_decoding_verification_23_gb300 import tree

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"spec_cache": sv.SpecCache, "spec_tree_args": sv.SpecTreeArgs, "spec_weigh_args": sv.SpecWeighArgs,
           "spec_evict_args": sv.SpecEvictArgs, "spec_commit_args": sv.SpecCommitArgs,
           "spec_beam_args": sv.SpecBeamArgs, "spec_beam_state": sv.SpecBeamState}


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return tree._lib()


def test_header_and_library_declare_the_python_names(lib):
    text = open(os.path.join(ROOT, "include", "spec_tree.h")).read()
    names = sorted(set(re.findall(r"^(?:size_t|int) (spec_\w+)\(", text, re.M)))
    assert names == sorted(sv.EXPORTED_TREE)
    out = subprocess.run(["nm", "-D", "--defined-only", sv.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r" T (spec_\w+)", out))


@pytest.mark.parametrize("name", sorted(STRUCTS))
def test_struct_layout_matches_header(tmp_path, name):
    cls = STRUCTS[name]
    body = "\n".join(f'  printf("{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spec_tree.h"\nint main(void) {\n' + body +
                   f'\n  printf("size %zu\\n", sizeof({name}));\n  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for f in cls._fields_:
        assert int(got[f[0]]) == getattr(cls, f[0]).offset, f[0]
    assert int(got["size"]) == ctypes.sizeof(cls)


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "spec_tree.h")).read()
    for n in ("SPEC_F16", "SPEC_STATUS_BAD_PAGE", "SPEC_STATUS_BAD_LEN"):
        assert int(re.search(rf"{n} = (\d+)", text).group(1)) == getattr(sv, n)
    for n in ("SPEC_MAX_TREE", "SPEC_MAX_BEAMS", "SPEC_MAX_STATES"):
        assert int(re.search(rf"#define {n} (\d+)", text).group(1)) == getattr(sv, n)


# Arguments whose pointers are never followed: every call below is refused.
PTR = 1 << 20


def _set(x, kw):
    for k, v in kw.items():
        obj, name = (x.cache, k[6:]) if k.startswith("cache_") else (x, k)
        assert name in [f[0] for f in obj._fields_]
        setattr(obj, name, v)
    return x


def _cache(x):
    c = x.cache
    c.k = c.v = PTR
    c.dtype, c.layers, c.num_pages, c.page_size, c.heads, c.dim = sv.SPEC_BF16, 1, 8, 16, 2, 64
    c.s_layer, c.s_page, c.s_slot, c.s_head = 0, 2048, 128, 64
    return x


def tree_args(**kw):
    a = _cache(sv.SpecTreeArgs())
    a.B, a.total_nodes, a.max_nodes, a.heads_q, a.scale = 2, 6, 4, 4, 0.125
    a.cu_nodes = a.q = a.k_new = a.v_new = a.block_table = a.ctx_len = PTR
    a.sq_node, a.sq_head, a.sn_node, a.sn_head, a.ld_table = 256, 64, 128, 64, 4
    return _set(a, kw)


CACHE_REFUSALS = [
    (dict(cache_k=None), sv.SPEC_ERR_NULL), (dict(cache_dtype=sv.SPEC_F32), sv.SPEC_ERR_DTYPE),
    (dict(cache_dtype=9), sv.SPEC_ERR_DTYPE), (dict(cache_layers=0), sv.SPEC_ERR_SHAPE),
    (dict(cache_num_pages=0), sv.SPEC_ERR_SHAPE), (dict(cache_page_size=0), sv.SPEC_ERR_SHAPE),
    (dict(cache_heads=0), sv.SPEC_ERR_SHAPE), (dict(cache_dim=80), sv.SPEC_ERR_SHAPE),
    (dict(cache_num_pages=1 << 28), sv.SPEC_ERR_SHAPE), (dict(cache_k=PTR + 8), sv.SPEC_ERR_ALIGN),
    (dict(cache_s_slot=68), sv.SPEC_ERR_ALIGN), (dict(cache_s_page=-8), sv.SPEC_ERR_ALIGN),
    (dict(cache_s_head=65), sv.SPEC_ERR_ALIGN), (dict(ld_table=0), sv.SPEC_ERR_SHAPE),
    (dict(ld_table=1 << 28), sv.SPEC_ERR_SHAPE), (dict(block_table=None), sv.SPEC_ERR_NULL), (dict(B=0), sv.SPEC_ERR_SHAPE),
]


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(cache_v=None), sv.SPEC_ERR_NULL), (dict(max_nodes=257), sv.SPEC_ERR_SHAPE),
    (dict(total_nodes=9), sv.SPEC_ERR_SHAPE), (dict(total_nodes=-1), sv.SPEC_ERR_SHAPE),
    (dict(heads_q=3), sv.SPEC_ERR_SHAPE), (dict(heads_q=0), sv.SPEC_ERR_SHAPE), (dict(layer=1), sv.SPEC_ERR_SHAPE),
    (dict(layer=-1), sv.SPEC_ERR_SHAPE), (dict(scale=float("nan")), sv.SPEC_ERR_SHAPE),
    (dict(scale=float("inf")), sv.SPEC_ERR_SHAPE), (dict(cu_nodes=None), sv.SPEC_ERR_NULL),
    (dict(ctx_len=None), sv.SPEC_ERR_NULL), (dict(q=None), sv.SPEC_ERR_NULL), (dict(v_new=None), sv.SPEC_ERR_NULL),
    (dict(q=PTR + 2), sv.SPEC_ERR_ALIGN), (dict(sq_head=60), sv.SPEC_ERR_ALIGN), (dict(sn_node=-8), sv.SPEC_ERR_ALIGN),
    (dict(tree_mask=PTR, mask_words=0), sv.SPEC_ERR_SHAPE),
])
def test_attention_refuses(lib, kw, code):
    a = tree_args(**kw)
    assert lib.spec_tree_attention(ctypes.byref(a), PTR, 256, 64, None, None, PTR, 1 << 40, None) == code
    assert lib.spec_tree_workspace_bytes(ctypes.byref(a)) == 0


def test_attention_refuses_its_buffers(lib):
    a = tree_args()
    n = lib.spec_tree_workspace_bytes(ctypes.byref(a))
    assert n > 0

    def call(out=PTR, so=256, ws=PTR, size=n):
        return lib.spec_tree_attention(ctypes.byref(a), out, so, 64, None, None, ws, size, None)

    assert call(out=None) == sv.SPEC_ERR_NULL
    assert call(out=PTR + 4) == sv.SPEC_ERR_ALIGN
    assert call(so=257) == sv.SPEC_ERR_ALIGN
    assert call(ws=None) == sv.SPEC_ERR_WORKSPACE
    assert call(ws=PTR + 128) == sv.SPEC_ERR_WORKSPACE
    assert call(size=n - 1) == sv.SPEC_ERR_WORKSPACE
    assert lib.spec_tree_attention(None, PTR, 256, 64, None, None, PTR, n, None) == sv.SPEC_ERR_NULL


def weigh_args(**kw):
    a = _cache(sv.SpecWeighArgs())
    a.B, a.total_rows, a.max_rows, a.heads_q, a.scale, a.ld, a.ld_table = 2, 6, 4, 4, 0.125, 64, 4
    a.cu_rows = a.q = a.lse = a.block_table = a.kv_len = PTR
    a.sq_row, a.sq_head = 256, 64
    return _set(a, kw)


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(total_rows=9), sv.SPEC_ERR_SHAPE), (dict(max_rows=-1), sv.SPEC_ERR_SHAPE), (dict(ld=0), sv.SPEC_ERR_SHAPE),
    (dict(heads_q=5), sv.SPEC_ERR_SHAPE), (dict(layer=2), sv.SPEC_ERR_SHAPE), (dict(lse=None), sv.SPEC_ERR_NULL),
    (dict(kv_len=None), sv.SPEC_ERR_NULL), (dict(cu_rows=None), sv.SPEC_ERR_NULL), (dict(sq_row=4), sv.SPEC_ERR_ALIGN),
    (dict(max_rows=1 << 30, total_rows=4), sv.SPEC_ERR_SHAPE), (dict(scale=float("nan")), sv.SPEC_ERR_SHAPE),
])
def test_weights_refuse(lib, kw, code):
    a = weigh_args(**kw)
    assert lib.spec_attention_weights(ctypes.byref(a), None, PTR, None, None) == code


def test_weights_refuse_no_output(lib):
    assert lib.spec_attention_weights(ctypes.byref(weigh_args()), None, None, None, None) == sv.SPEC_ERR_NULL


def evict_args(**kw):
    a = _cache(sv.SpecEvictArgs())
    a.B, a.keep, a.sink, a.recent, a.ld, a.ld_table, a.ld_to = 2, 32, 4, 8, 64, 4, 2
    a.weights = a.kv_len = a.block_table = a.to_table = PTR
    return _set(a, kw)


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(keep=0), sv.SPEC_ERR_SHAPE), (dict(sink=30), sv.SPEC_ERR_SHAPE), (dict(recent=-1), sv.SPEC_ERR_SHAPE),
    (dict(sink=-1), sv.SPEC_ERR_SHAPE), (dict(ld_to=1), sv.SPEC_ERR_SHAPE), (dict(ld=0), sv.SPEC_ERR_SHAPE),
    (dict(layer=1), sv.SPEC_ERR_SHAPE), (dict(weights=None), sv.SPEC_ERR_NULL), (dict(to_table=None), sv.SPEC_ERR_NULL),
    (dict(kv_len=None), sv.SPEC_ERR_NULL),
])
def test_eviction_refuses(lib, kw, code):
    assert lib.spec_cache_evict(ctypes.byref(evict_args(**kw)), PTR, None, PTR, None, None) == code


def commit_args(**kw):
    a = _cache(sv.SpecCommitArgs())
    a.B, a.total_nodes, a.ld_path, a.ld_table = 2, 6, 4, 4
    a.cu_nodes = a.k_new = a.v_new = a.path = a.path_len = a.block_table = a.ctx_len = PTR
    a.sn_layer, a.sn_node, a.sn_head = 1024, 128, 64
    return _set(a, kw)


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(ld_path=0), sv.SPEC_ERR_SHAPE), (dict(total_nodes=-1), sv.SPEC_ERR_SHAPE), (dict(path=None), sv.SPEC_ERR_NULL),
    (dict(path_len=None), sv.SPEC_ERR_NULL), (dict(k_new=None), sv.SPEC_ERR_NULL), (dict(k_new=PTR + 8), sv.SPEC_ERR_ALIGN),
    (dict(sn_layer=4), sv.SPEC_ERR_ALIGN), (dict(cache_layers=70000), sv.SPEC_ERR_SHAPE),
])
def test_commit_refuses(lib, kw, code):
    assert lib.spec_cache_commit(ctypes.byref(commit_args(**kw)), PTR, None, None) == code


def beam_args(**kw):
    a = sv.SpecBeamArgs()
    a.B, a.W, a.keep, a.V, a.dtype, a.ld = 2, 3, 4, 1000, sv.SPEC_BF16, 1000
    a.logits = a.scores = PTR
    return _set(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=sv.SPEC_F16), sv.SPEC_ERR_DTYPE), (dict(B=0), sv.SPEC_ERR_SHAPE), (dict(W=65), sv.SPEC_ERR_SHAPE),
    (dict(keep=65), sv.SPEC_ERR_SHAPE), (dict(keep=0), sv.SPEC_ERR_SHAPE), (dict(V=0), sv.SPEC_ERR_SHAPE),
    (dict(ld=999), sv.SPEC_ERR_SHAPE), (dict(ld=1001), sv.SPEC_ERR_ALIGN), (dict(logits=PTR + 2), sv.SPEC_ERR_ALIGN),
    (dict(logits=None), sv.SPEC_ERR_NULL), (dict(scores=None), sv.SPEC_ERR_NULL),
    (dict(finished=PTR, end_token=1000), sv.SPEC_ERR_SHAPE), (dict(finished=PTR, end_token=-1), sv.SPEC_ERR_SHAPE),
    (dict(V=2 ** 30, ld=2 ** 30), sv.SPEC_ERR_SHAPE),
])
def test_beams_refuse(lib, kw, code):
    a = beam_args(**kw)
    assert lib.spec_beam_select(ctypes.byref(a), PTR, PTR, PTR, None, PTR, 1 << 40, None) == code
    assert lib.spec_beam_workspace_bytes(ctypes.byref(a)) == 0


def test_beams_refuse_their_buffers(lib):
    a = beam_args()
    n = lib.spec_beam_workspace_bytes(ctypes.byref(a))
    assert lib.spec_beam_select(ctypes.byref(a), PTR, PTR, None, None, PTR, n, None) == sv.SPEC_ERR_NULL
    assert lib.spec_beam_select(ctypes.byref(a), PTR, PTR, PTR, None, PTR, n - 1, None) == sv.SPEC_ERR_WORKSPACE
    assert lib.spec_beam_select(ctypes.byref(a), PTR, PTR, PTR, None, PTR + 16, n, None) == sv.SPEC_ERR_WORKSPACE


def test_reordering_refuses(lib):
    s = sv.SpecBeamState()
    s.src = s.dst = PTR
    s.row_bytes, s.outer = 64, 1
    block = (sv.SpecBeamState * 9)(*[s] * 9)
    assert lib.spec_beam_reorder(2, 3, 4, None, block, 1, None) == sv.SPEC_ERR_NULL
    assert lib.spec_beam_reorder(2, 3, 4, PTR, None, 1, None) == sv.SPEC_ERR_NULL
    assert lib.spec_beam_reorder(2, 3, 4, PTR, block, 9, None) == sv.SPEC_ERR_SHAPE
    assert lib.spec_beam_reorder(0, 3, 4, PTR, block, 1, None) == sv.SPEC_ERR_SHAPE
    block[0].dst = None
    assert lib.spec_beam_reorder(2, 3, 4, PTR, block, 1, None) == sv.SPEC_ERR_NULL
    block[0].dst, block[0].row_bytes = PTR, -1
    assert lib.spec_beam_reorder(2, 3, 4, PTR, block, 1, None) == sv.SPEC_ERR_SHAPE


def test_no_device_is_an_error(lib):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    a, e, c, b = tree_args(), evict_args(), commit_args(), beam_args()
    n, m = lib.spec_tree_workspace_bytes(ctypes.byref(a)), lib.spec_beam_workspace_bytes(ctypes.byref(b))
    assert lib.spec_tree_attention(ctypes.byref(a), PTR, 256, 64, None, None, PTR, n, None) == sv.SPEC_ERR_DEVICE
    assert lib.spec_attention_weights(ctypes.byref(weigh_args()), None, PTR, None, None) == sv.SPEC_ERR_DEVICE
    assert lib.spec_cache_evict(ctypes.byref(e), PTR, None, PTR, None, None) == sv.SPEC_ERR_DEVICE
    assert lib.spec_cache_commit(ctypes.byref(c), PTR, None, None) == sv.SPEC_ERR_DEVICE
    assert lib.spec_beam_select(ctypes.byref(b), PTR, PTR, PTR, None, PTR, m, None) == sv.SPEC_ERR_DEVICE


def test_tensor_checks_refuse():
    import torch

    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        sv.make_cache(k, k)                      # not on a GPU
    with pytest.raises(TypeError):
        sv.make_cache(k.float(), k.float())
    with pytest.raises(TypeError):
        sv.make_beam_args(logits=torch.zeros(4, 8), V=8, scores=torch.zeros(2, 2), keep=2)
    with pytest.raises(TypeError):
        sv.make_reorder_args(parents=torch.zeros(2, 2, dtype=torch.int32), beams=2, states=[])
