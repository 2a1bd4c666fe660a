"""Operators beside the drafted-tree ones (C ABI in ``include/spec_serve.h``):
norms with the position rotation, attention with a sliding window, and
attention over and commitment to a cache held in 8 bits.

As in ``tree``: ``make_*`` builds an argument block from CUDA tensors once; the
calls take it, with the results' buffers where the caller keeps them.
"""
from __future__ import annotations

import ctypes

from . import _check_f32, _check_i32, _ptr, load_library
from .tree import (SpecTreeArgs, _check_lengths, _check_out, _check_shape, _check_table, _check_vectors,
                   _device, _empty, _f32, _i32, _i64, _int32, _kv_dtype, _p, _raise, _stream_handle, _workspace_bytes,
                   make_tree_args)

EXPORTED_SERVE = ("spec_norm_rotate", "spec_window_workspace_bytes", "spec_window_attention",
                  "spec_cache8_workspace_bytes", "spec_cache8_attention", "spec_cache8_commit")


class SpecRotateArgs(ctypes.Structure):
    """Mirror of ``spec_rotate_args``."""

    _fields_ = [("rows", _i32), ("heads_q", _i32), ("heads_k", _i32), ("dim", _i32), ("rot", _i32),
                ("interleaved", _i32), ("dtype", _i32), ("eps", _f32), ("q", _p), ("sq_row", _i64), ("sq_head", _i64),
                ("k", _p), ("sk_row", _i64), ("sk_head", _i64), ("q_weight", _p), ("k_weight", _p), ("positions", _p),
                ("inv_freq", _p)]


class SpecWindowArgs(ctypes.Structure):
    """Mirror of ``spec_window_args``."""

    _fields_ = [("tree", SpecTreeArgs), ("window", _i32), ("sinks", _i32)]


class SpecCache8(ctypes.Structure):
    """Mirror of ``spec_cache8``."""

    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("layers", _i32), ("num_pages", _i32),
                ("page_size", _i32), ("heads", _i32), ("dim", _i32), ("block", _i32), ("s_layer", _i64),
                ("s_page", _i64), ("s_slot", _i64), ("s_head", _i64), ("c_layer", _i64), ("c_page", _i64),
                ("c_block", _i64), ("c_head", _i64)]


class SpecCache8Args(ctypes.Structure):
    """Mirror of ``spec_cache8_args``."""

    _fields_ = [("B", _i32), ("total_nodes", _i32), ("max_nodes", _i32), ("heads_q", _i32), ("layer", _i32),
                ("scale", _f32), ("dtype", _i32), ("window", _i32), ("sinks", _i32), ("mask_words", _i32),
                ("cu_nodes", _p), ("q", _p), ("sq_node", _i64), ("sq_head", _i64), ("k_new", _p), ("v_new", _p),
                ("sn_node", _i64), ("sn_head", _i64), ("tree_mask", _p), ("cache", SpecCache8), ("block_table", _p),
                ("ctx_len", _p), ("ld_table", _i32), ("pad", _i32)]


class SpecCache8CommitArgs(ctypes.Structure):
    """Mirror of ``spec_cache8_commit_args``."""

    _fields_ = [("B", _i32), ("total_nodes", _i32), ("dtype", _i32), ("ld_path", _i32), ("cu_nodes", _p),
                ("k_new", _p), ("v_new", _p), ("sn_layer", _i64), ("sn_node", _i64), ("sn_head", _i64), ("path", _p),
                ("path_len", _p), ("cache", SpecCache8), ("block_table", _p), ("ctx_len", _p), ("ld_table", _i32),
                ("pad", _i32)]


_declared = None


def _lib():
    global _declared
    lib = load_library()
    if _declared is lib:
        return lib
    c_int, size_t, P = ctypes.c_int, ctypes.c_size_t, ctypes.POINTER
    lib.spec_norm_rotate.restype = c_int
    lib.spec_norm_rotate.argtypes = [P(SpecRotateArgs), _p, _i64, _i64, _p, _i64, _i64, _p]
    for name, block in (("window", SpecWindowArgs), ("cache8", SpecCache8Args)):
        f = getattr(lib, f"spec_{name}_workspace_bytes")
        f.restype, f.argtypes = size_t, [P(block)]
        f = getattr(lib, f"spec_{name}_attention")
        f.restype, f.argtypes = c_int, [P(block), _p, _i64, _i64, _p, _p, _p, size_t, _p]
    lib.spec_cache8_commit.restype = c_int
    lib.spec_cache8_commit.argtypes = [P(SpecCache8CommitArgs), _p, _p, _p]
    _declared = lib
    return lib


# ---------------------------------------------------- norms and positions

def make_rotate_args(*, q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                     interleaved: bool = False) -> SpecRotateArgs:
    """``spec_rotate_args``: q [rows, heads_q, dim] and k [rows, heads_k, dim] of any strides with a unit inner one
    (either may be None), positions [rows] int32, inv_freq [pairs] float32 (twice as many channels turn), weights
    [dim] of the same type (None: ones)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is needed")
    a = SpecRotateArgs()
    a.dtype = _kv_dtype(x)
    _check_i32("positions", positions)
    _check_f32("inv_freq", inv_freq)
    if inv_freq.dim() != 1:
        raise ValueError(f"inv_freq must have one axis, got {tuple(inv_freq.shape)}")
    a.rows, a.dim = x.shape[0], x.shape[-1]
    _check_shape("positions", positions, (a.rows,))
    for name, t, w in (("q", q, q_weight), ("k", k, k_weight)):
        if t is not None:
            _check_vectors(name, t, 3, x.dtype)
            _check_shape(name, t, (a.rows, t.shape[1], a.dim))
            setattr(a, f"heads_{name}", t.shape[1])
            setattr(a, name, _ptr(t))
            setattr(a, f"s{name}_row", t.stride(0))
            setattr(a, f"s{name}_head", t.stride(1))
        if w is not None:
            _check_vectors(f"{name}_weight", w, 1, x.dtype)
            _check_shape(f"{name}_weight", w, (a.dim,))
            setattr(a, f"{name}_weight", _ptr(w))
    a.rot, a.interleaved, a.eps = 2 * inv_freq.numel(), int(bool(interleaved)), float(eps)
    a.positions, a.inv_freq = _ptr(positions), _ptr(inv_freq)
    a._keep = (q, k, positions, inv_freq, q_weight, k_weight)
    a.torch_dtype = x.dtype
    return a


def spec_norm_rotate(args: SpecRotateArgs, *, out_q=None, out_k=None, stream=None):
    """Normed and rotated queries and keys through ``spec_norm_rotate``.  Returns (q [rows, heads_q, dim], k [rows,
    heads_k, dim]), None for one that the block does not have.  Results may have any strides with a unit inner one
    and rows and heads that do not overlap; they may be the inputs themselves."""
    got = []
    for name, out, heads in (("out_q", out_q, args.heads_q), ("out_k", out_k, args.heads_k)):
        shape = (args.rows, heads, args.dim)
        if out is not None:
            _check_vectors(name, out, 3, args.torch_dtype)
            _check_shape(name, out, shape)
        elif heads > 0:
            out = _empty(stream, *shape, dtype=args.torch_dtype, like=_device())
        got.append(out)
    sides = [x for out in got for x in ((_ptr(out), out.stride(0), out.stride(1)) if out is not None else (None, 0, 0))]
    rc = _lib().spec_norm_rotate(ctypes.byref(args), *sides, _stream_handle(stream))
    _raise(rc, "spec_norm_rotate")
    return got[0], got[1]


# --------------------------------------------------------------- attention

def _attend(name, args, B, total, heads_q, dim, workspace, out, out_lse, out_status, stream):
    import torch

    lib = _lib()
    if workspace is None:
        workspace = _make_workspace(name, args, stream)
    ws_bytes = _workspace_bytes(workspace)
    shape = (total, heads_q, dim)
    if out is None:
        out = _empty(stream, *shape, dtype=args.torch_dtype, like=workspace.device)
    else:
        _check_vectors("out", out, 3, args.torch_dtype)
        _check_shape("out", out, shape)
    if out_lse is None:
        out_lse = _empty(stream, *shape[:2], dtype=torch.float32, like=workspace.device)
    else:
        _check_out("out_lse", out_lse, shape[:2], torch.float32)
    if out_status is None:
        out_status = _empty(stream, B, dtype=torch.int32, like=workspace.device)
    else:
        _check_out("out_status", out_status, (B,), torch.int32)
    rc = getattr(lib, f"spec_{name}_attention")(ctypes.byref(args), _ptr(out), out.stride(0), out.stride(1),
                                                _ptr(out_lse), _ptr(out_status), _ptr(workspace), ws_bytes,
                                                _stream_handle(stream))
    _raise(rc, f"spec_{name}_attention")
    return out, out_lse, out_status


def _make_workspace(name, args, stream):
    import torch

    n = int(getattr(_lib(), f"spec_{name}_workspace_bytes")(ctypes.byref(args)))
    return _empty(stream, max(n, 256), dtype=torch.uint8, like=_device())


def make_window_args(*, window: int, sinks: int = 0, **tree) -> SpecWindowArgs:
    """``spec_window_args``: what ``make_tree_args`` takes, and the tokens that a row still sees, the last `window` and
    the first `sinks` of its own text."""
    t = make_tree_args(**tree)
    a = SpecWindowArgs()
    a.tree = t
    a.window, a.sinks = _int32("window", window), _int32("sinks", sinks)
    a._keep = t._keep
    a.torch_dtype = t.torch_dtype
    return a


def spec_window_workspace_bytes(args: SpecWindowArgs) -> int:
    return int(_lib().spec_window_workspace_bytes(ctypes.byref(args)))


def make_window_workspace(args: SpecWindowArgs, stream=None):
    return _make_workspace("window", args, stream)


def spec_window_attention(args: SpecWindowArgs, *, workspace=None, out=None, out_lse=None, out_status=None,
                          stream=None):
    """Attention of drafted trees with a sliding window and sinks through ``spec_window_attention``.  Returns (out
    [nodes, heads_q, dim], lse [nodes, heads_q] float32, status [B] int32)."""
    t = args.tree
    return _attend("window", args, t.B, t.total_nodes, t.heads_q, t.cache.dim, workspace, out, out_lse, out_status,
                   stream)


# -------------------------------------------------------------- 8-bit cache

def make_cache8(k, v, k_scale, v_scale) -> SpecCache8:
    """``spec_cache8``: two float8_e4m3fn tensors [pages, page_size, heads, dim] or [layers, pages, page_size, heads,
    dim], of any strides (the same in both) with a unit inner one, and their float32 scales [pages, blocks, heads] or
    [layers, pages, blocks, heads] (the same strides in both): a page has `blocks` blocks of tokens of a scale each."""
    import torch

    if k.dim() not in (4, 5):
        raise TypeError("a cache has 4 axes (pages, slots, heads, channels), or 5 with its layers before them")
    for name, t in (("k", k), ("v", v)):
        _check_vectors(name, t, k.dim(), torch.float8_e4m3fn)
    if k.shape != v.shape or k.stride() != v.stride():
        raise ValueError("keys and values must have the same shape and strides")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t.dim() != k.dim() - 1 or t.dtype != torch.float32 or not t.is_cuda:
            raise TypeError(f"{name} must be a {k.dim() - 1}-D float32 CUDA tensor")
    if k_scale.shape != v_scale.shape or k_scale.stride() != v_scale.stride():
        raise ValueError("the scales of keys and values must have the same shape and strides")
    if k.dim() == 4:
        shape, stride = (1, *k.shape), (0, *k.stride())
        blocks, at = (1, *k_scale.shape), (0, *k_scale.stride())
    else:
        shape, stride, blocks, at = tuple(k.shape), tuple(k.stride()), tuple(k_scale.shape), tuple(k_scale.stride())
    layers, pages, page, heads, dim = shape
    if blocks[:2] != (layers, pages) or blocks[3] != heads or blocks[2] < 1 or page % max(1, blocks[2]) != 0:
        raise ValueError(f"scales of a cache of shape {tuple(k.shape)} must have shape ({'layers, ' * (k.dim() - 4)}pages, "
                         f"blocks, heads) with blocks that divide {page}, got {tuple(k_scale.shape)}")
    c = SpecCache8()
    c.k, c.v, c.k_scale, c.v_scale = _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale)
    c.layers, c.num_pages, c.page_size, c.heads, c.dim = shape
    c.block = page // blocks[2]
    c.s_layer, c.s_page, c.s_slot, c.s_head = stride[:4]
    c.c_layer, c.c_page, c.c_block, c.c_head = at
    c._keep = (k, v, k_scale, v_scale)
    return c


def make_cache8_args(*, q, k_new, v_new, cu_nodes, max_nodes: int, cache: SpecCache8, block_table, ctx_len,
                     tree_mask=None, scale=None, layer: int = 0, window: int = 0, sinks: int = 0) -> SpecCache8Args:
    """``spec_cache8_args``: as ``make_tree_args`` with an 8-bit cache; a `window` (0: none) and `sinks` as in
    ``make_window_args``."""
    a = SpecCache8Args()
    a.dtype = _kv_dtype(q)
    for name, t in (("q", q), ("k_new", k_new), ("v_new", v_new)):
        _check_vectors(name, t, 3, q.dtype)
    _check_i32("cu_nodes", cu_nodes)
    B, total = cu_nodes.numel() - 1, q.shape[0]
    _check_shape("q", q, (total, q.shape[1], cache.dim))
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _check_shape(name, t, (total, cache.heads, cache.dim))
    if total > 0 and k_new.stride() != v_new.stride():
        raise ValueError("k_new and v_new must have the same strides")
    _check_table("block_table", block_table, B)
    _check_lengths("ctx_len", ctx_len, B)
    if tree_mask is not None:
        _check_i32("tree_mask", tree_mask)
        if tree_mask.dim() != 2 or tree_mask.shape[0] != total:
            raise ValueError(f"tree_mask must have shape ({total}, words), got {tuple(tree_mask.shape)}")
        a.tree_mask, a.mask_words = _ptr(tree_mask), tree_mask.shape[1]
    a.B, a.total_nodes, a.max_nodes, a.heads_q = B, total, _int32("max_nodes", max_nodes), q.shape[1]
    a.layer = _int32("layer", layer)
    a.window, a.sinks = _int32("window", window), _int32("sinks", sinks)
    a.scale = cache.dim ** -0.5 if scale is None else float(scale)
    a.cu_nodes, a.q, a.k_new, a.v_new = _ptr(cu_nodes), _ptr(q), _ptr(k_new), _ptr(v_new)
    a.sq_node, a.sq_head = q.stride()[:2]
    a.sn_node, a.sn_head = k_new.stride()[:2]
    a.cache = cache
    a.block_table, a.ld_table, a.ctx_len = _ptr(block_table), block_table.shape[1], _ptr(ctx_len)
    a._keep = (q, k_new, v_new, cu_nodes, cache, cache._keep, block_table, ctx_len, tree_mask)
    a.torch_dtype = q.dtype
    return a


def spec_cache8_workspace_bytes(args: SpecCache8Args) -> int:
    return int(_lib().spec_cache8_workspace_bytes(ctypes.byref(args)))


def make_cache8_workspace(args: SpecCache8Args, stream=None):
    return _make_workspace("cache8", args, stream)


def spec_cache8_attention(args: SpecCache8Args, *, workspace=None, out=None, out_lse=None, out_status=None,
                          stream=None):
    """Attention of drafted trees over an 8-bit cache through ``spec_cache8_attention``.  Returns (out [nodes, heads_q,
    dim], lse [nodes, heads_q] float32, status [B] int32)."""
    return _attend("cache8", args, args.B, args.total_nodes, args.heads_q, args.cache.dim, workspace, out, out_lse,
                   out_status, stream)


def make_cache8_commit_args(*, k_new, v_new, cu_nodes, path, path_len, cache: SpecCache8, block_table,
                            ctx_len) -> SpecCache8CommitArgs:
    """``spec_cache8_commit_args``: k_new and v_new [layers, nodes, heads, dim] (or [nodes, heads, dim] for a cache of
    one layer), path [B, length] int32 nodes of each request, path_len [B]."""
    if k_new.dim() == 3:
        k_new, v_new = k_new[None], v_new[None]
    a = SpecCache8CommitArgs()
    a.dtype = _kv_dtype(k_new)
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _check_vectors(name, t, 4, k_new.dtype)
        _check_shape(name, t, (cache.layers, k_new.shape[1], cache.heads, cache.dim))
    if k_new.numel() > 0 and k_new.stride() != v_new.stride():
        raise ValueError("k_new and v_new must have the same strides")
    _check_i32("cu_nodes", cu_nodes)
    B = cu_nodes.numel() - 1
    _check_table("path", path, B)
    _check_lengths("path_len", path_len, B)
    _check_table("block_table", block_table, B)
    _check_lengths("ctx_len", ctx_len, B)
    a.B, a.total_nodes, a.cu_nodes = B, k_new.shape[1], _ptr(cu_nodes)
    a.k_new, a.v_new = _ptr(k_new), _ptr(v_new)
    a.sn_layer, a.sn_node, a.sn_head = k_new.stride()[:3]
    a.path, a.path_len, a.cache = _ptr(path), _ptr(path_len), cache
    a.block_table, a.ctx_len = _ptr(block_table), _ptr(ctx_len)
    a.ld_path, a.ld_table = path.shape[1], block_table.shape[1]
    a._keep = (k_new, v_new, cu_nodes, path, path_len, cache, cache._keep, block_table, ctx_len)
    return a


def spec_cache8_commit(args: SpecCache8CommitArgs, *, out_len=None, out_status=None, stream=None):
    """Writes the accepted paths' keys and values to an 8-bit cache through ``spec_cache8_commit``.  Returns (new
    lengths [B] int32, status [B]).  `out_len` may be the block's ctx_len."""
    import torch

    got = []
    for name, t in (("out_len", out_len), ("out_status", out_status)):
        _check_out(name, t, (args.B,), torch.int32)
        got.append(_empty(stream, args.B, dtype=torch.int32, like=_device()) if t is None else t)
    rc = _lib().spec_cache8_commit(ctypes.byref(args), _ptr(got[0]), _ptr(got[1]), _stream_handle(stream))
    _raise(rc, "spec_cache8_commit")
    return got[0], got[1]
