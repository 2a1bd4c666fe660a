"""Drafted-tree operators over a paged cache (C ABI in ``include/spec_tree.h``).

``make_*`` builds an argument block from CUDA tensors once; the calls take
it, with the results' buffers where the caller keeps them.  A block holds the
tensors it points to.  Work is enqueued on ``stream`` (the current one by
default); buffers that a call allocates itself belong to that stream.
"""
from __future__ import annotations

import ctypes

from . import SPEC_BF16, SPEC_OK, SpecError, _check_f32, _check_i32, _dtype_code, _ptr, load_library

SPEC_F16 = 2
SPEC_STATUS_BAD_PAGE = 32
SPEC_STATUS_BAD_LEN = 64
SPEC_MAX_TREE = 256
SPEC_MAX_BEAMS = 64
SPEC_MAX_STATES = 8

EXPORTED_TREE = ("spec_tree_workspace_bytes", "spec_tree_attention", "spec_attention_weights", "spec_cache_evict",
                 "spec_cache_commit", "spec_beam_workspace_bytes", "spec_beam_select", "spec_beam_reorder")

_i32, _i64, _f32, _p = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class SpecCache(ctypes.Structure):
    """Mirror of ``spec_cache``."""

    _fields_ = [("k", _p), ("v", _p), ("dtype", _i32), ("layers", _i32), ("num_pages", _i32), ("page_size", _i32),
                ("heads", _i32), ("dim", _i32), ("s_layer", _i64), ("s_page", _i64), ("s_slot", _i64),
                ("s_head", _i64)]


class SpecTreeArgs(ctypes.Structure):
    """Mirror of ``spec_tree_args``."""

    _fields_ = [("B", _i32), ("total_nodes", _i32), ("max_nodes", _i32), ("heads_q", _i32), ("layer", _i32),
                ("scale", _f32), ("cu_nodes", _p), ("q", _p), ("sq_node", _i64), ("sq_head", _i64), ("k_new", _p),
                ("v_new", _p), ("sn_node", _i64), ("sn_head", _i64), ("tree_mask", _p), ("mask_words", _i32),
                ("ld_table", _i32), ("cache", SpecCache), ("block_table", _p), ("ctx_len", _p)]


class SpecWeighArgs(ctypes.Structure):
    """Mirror of ``spec_weigh_args``."""

    _fields_ = [("B", _i32), ("total_rows", _i32), ("max_rows", _i32), ("heads_q", _i32), ("layer", _i32),
                ("scale", _f32), ("cu_rows", _p), ("q", _p), ("sq_row", _i64), ("sq_head", _i64), ("lse", _p),
                ("cache", SpecCache), ("block_table", _p), ("kv_len", _p), ("ld_table", _i32), ("ld", _i32)]


class SpecEvictArgs(ctypes.Structure):
    """Mirror of ``spec_evict_args``."""

    _fields_ = [("B", _i32), ("keep", _i32), ("sink", _i32), ("recent", _i32), ("layer", _i32), ("ld", _i32),
                ("weights", _p), ("kv_len", _p), ("cache", SpecCache), ("block_table", _p), ("to_table", _p),
                ("ld_table", _i32), ("ld_to", _i32)]


class SpecCommitArgs(ctypes.Structure):
    """Mirror of ``spec_commit_args``."""

    _fields_ = [("B", _i32), ("total_nodes", _i32), ("cu_nodes", _p), ("k_new", _p), ("v_new", _p),
                ("sn_layer", _i64), ("sn_node", _i64), ("sn_head", _i64), ("path", _p), ("path_len", _p),
                ("cache", SpecCache), ("block_table", _p), ("ctx_len", _p), ("ld_path", _i32), ("ld_table", _i32)]


class SpecBeamArgs(ctypes.Structure):
    """Mirror of ``spec_beam_args``."""

    _fields_ = [("B", _i32), ("W", _i32), ("keep", _i32), ("V", _i32), ("dtype", _i32), ("end_token", _i32),
                ("logits", _p), ("ld", _i64), ("scores", _p), ("finished", _p)]


class SpecBeamState(ctypes.Structure):
    """Mirror of ``spec_beam_state``."""

    _fields_ = [("src", _p), ("dst", _p), ("row_bytes", _i64), ("src_outer", _i64), ("src_batch", _i64),
                ("src_beam", _i64), ("dst_outer", _i64), ("dst_batch", _i64), ("dst_beam", _i64), ("outer", _i32),
                ("pad", _i32)]


class ReorderArgs:
    """The arguments of ``spec_beam_reorder``."""

    def __init__(self, B, W, keep, parents, states, keep_alive):
        self.B, self.W, self.keep = B, W, keep
        self.parents = _ptr(parents)
        self.states = states
        self._keep = keep_alive


_declared = None


def _lib():
    global _declared
    lib = load_library()
    if _declared is lib:
        return lib
    c_int, size_t, P = ctypes.c_int, ctypes.c_size_t, ctypes.POINTER
    lib.spec_tree_workspace_bytes.restype = size_t
    lib.spec_tree_workspace_bytes.argtypes = [P(SpecTreeArgs)]
    lib.spec_tree_attention.restype = c_int
    lib.spec_tree_attention.argtypes = [P(SpecTreeArgs), _p, _i64, _i64, _p, _p, _p, size_t, _p]
    lib.spec_attention_weights.restype = c_int
    lib.spec_attention_weights.argtypes = [P(SpecWeighArgs), _p, _p, _p, _p]
    lib.spec_cache_evict.restype = c_int
    lib.spec_cache_evict.argtypes = [P(SpecEvictArgs), _p, _p, _p, _p, _p]
    lib.spec_cache_commit.restype = c_int
    lib.spec_cache_commit.argtypes = [P(SpecCommitArgs), _p, _p, _p]
    lib.spec_beam_workspace_bytes.restype = size_t
    lib.spec_beam_workspace_bytes.argtypes = [P(SpecBeamArgs)]
    lib.spec_beam_select.restype = c_int
    lib.spec_beam_select.argtypes = [P(SpecBeamArgs), _p, _p, _p, _p, _p, size_t, _p]
    lib.spec_beam_reorder.restype = c_int
    lib.spec_beam_reorder.argtypes = [_i32, _i32, _i32, _p, P(SpecBeamState), _i32, _p]
    _declared = lib
    return lib


# ----------------------------------------------------------------- helpers

def _raise(rc, where):
    if rc != SPEC_OK:
        raise SpecError(rc, where)


def _int32(name, x) -> int:
    """A whole number that its field holds: ctypes keeps the low 32 bits of
    any."""
    x = int(x)
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _stream_handle(stream) -> int:
    """The stream's handle; the current one is asked for without building the
    Python object around it, which costs more than a launch."""
    import torch

    if stream is not None:
        return int(stream.cuda_stream)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return int(torch.cuda.current_stream().cuda_stream)
    return raw(torch._C._cuda_getDevice())


def _empty(stream, *shape, dtype, like):
    """A buffer on `like`'s device that belongs to the stream of the call."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like)


def _device():
    import torch

    return torch.device("cuda", torch.cuda.current_device())


def _check_out(name, t, shape, dtype):
    """A caller's buffer: contiguous, of this shape and type."""
    if t is None:
        return
    if t.shape != shape or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}")


def _workspace_bytes(t):
    """The size of a caller's workspace, of any type."""
    if not t.is_cuda or not t.is_contiguous():
        raise TypeError("a workspace must be a contiguous CUDA tensor")
    return t.numel() * t.element_size()


def _kv_dtype(t):
    import torch

    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float16:
        return SPEC_F16
    raise TypeError(f"keys, values and queries must be bf16 or fp16, got {t.dtype}")


def _check_vectors(name, t, dims, dtype):
    if t.dim() != dims or t.dtype != dtype or not t.is_cuda or (t.numel() > 0 and t.stride(-1) != 1):
        raise TypeError(f"{name} must be a {dims}-D CUDA tensor of {dtype} with unit inner stride")


def _check_shape(name, t, shape):
    if t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_lengths(name, t, n):
    _check_i32(name, t)
    _check_shape(name, t, (n,))


def _check_table(name, t, B):
    _check_i32(name, t)
    if t.dim() != 2 or t.shape[0] != B:
        raise ValueError(f"{name} must have shape ({B}, pages), got {tuple(t.shape)}")


def make_cache(k, v) -> SpecCache:
    """``spec_cache`` of two tensors [pages, page_size, heads, dim] or
    [layers, pages, page_size, heads, dim], of any strides (the same in both)
    with a unit inner one."""
    dtype = _kv_dtype(k)
    if k.dim() not in (4, 5):
        raise TypeError("a cache has 4 axes (pages, slots, heads, channels), or 5 with its layers before them")
    for name, t in (("k", k), ("v", v)):
        _check_vectors(name, t, k.dim(), k.dtype)
    if k.shape != v.shape or k.stride() != v.stride():
        raise ValueError("keys and values must have the same shape and strides")
    c = SpecCache()
    c.k, c.v, c.dtype = _ptr(k), _ptr(v), dtype
    shape, stride = tuple(k.shape), tuple(k.stride())
    if k.dim() == 4:
        shape, stride = (1, *shape), (0, *stride)
    c.layers, c.num_pages, c.page_size, c.heads, c.dim = shape
    c.s_layer, c.s_page, c.s_slot, c.s_head = stride[:4]
    c._keep = (k, v)
    c.torch_dtype = k.dtype
    return c


# ---------------------------------------------------------- tree attention

def make_tree_args(*, q, k_new, v_new, cu_nodes, max_nodes: int, cache: SpecCache, block_table, ctx_len,
                   tree_mask=None, scale=None, layer: int = 0) -> SpecTreeArgs:
    """``spec_tree_args``: q [nodes, heads_q, dim], k_new and v_new [nodes,
    heads, dim] (their strides alike), cu_nodes [B+1], block_table [B, pages],
    ctx_len [B], tree_mask [nodes, words] int32 bits (None: chains).  `scale`
    is dim**-0.5 by default."""
    for name, t in (("q", q), ("k_new", k_new), ("v_new", v_new)):
        _check_vectors(name, t, 3, cache.torch_dtype)
    _check_i32("cu_nodes", cu_nodes)
    B, total = cu_nodes.numel() - 1, q.shape[0]
    _check_shape("q", q, (total, q.shape[1], cache.dim))
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _check_shape(name, t, (total, cache.heads, cache.dim))
    if total > 0 and k_new.stride() != v_new.stride():
        raise ValueError("k_new and v_new must have the same strides")
    _check_table("block_table", block_table, B)
    _check_lengths("ctx_len", ctx_len, B)
    a = SpecTreeArgs()
    if tree_mask is not None:
        _check_i32("tree_mask", tree_mask)
        if tree_mask.dim() != 2 or tree_mask.shape[0] != total:
            raise ValueError(f"tree_mask must have shape ({total}, words), got {tuple(tree_mask.shape)}")
        a.tree_mask, a.mask_words = _ptr(tree_mask), tree_mask.shape[1]
    a.B, a.total_nodes, a.max_nodes, a.heads_q = B, total, _int32("max_nodes", max_nodes), q.shape[1]
    a.layer = _int32("layer", layer)
    a.scale = cache.dim ** -0.5 if scale is None else float(scale)
    a.cu_nodes, a.q, a.k_new, a.v_new = _ptr(cu_nodes), _ptr(q), _ptr(k_new), _ptr(v_new)
    a.sq_node, a.sq_head = q.stride()[:2]
    a.sn_node, a.sn_head = k_new.stride()[:2]
    a.cache = cache
    a.block_table, a.ld_table, a.ctx_len = _ptr(block_table), block_table.shape[1], _ptr(ctx_len)
    a._keep = (q, k_new, v_new, cu_nodes, cache, block_table, ctx_len, tree_mask)
    a.torch_dtype = cache.torch_dtype
    return a


def spec_tree_workspace_bytes(args: SpecTreeArgs) -> int:
    return int(_lib().spec_tree_workspace_bytes(ctypes.byref(args)))


def make_tree_workspace(args: SpecTreeArgs, stream=None):
    import torch

    return _empty(stream, max(spec_tree_workspace_bytes(args), 256), dtype=torch.uint8, like=_device())


def spec_tree_attention(args: SpecTreeArgs, *, workspace=None, out=None, out_lse=None, out_status=None, stream=None):
    """Attention of drafted trees over a paged cache through
    ``spec_tree_attention``.  Returns (out [nodes, heads_q, dim], lse [nodes,
    heads_q] float32, status [B] int32).  `out` may have any strides with a
    unit inner one."""
    import torch

    lib = _lib()
    shape = (args.total_nodes, args.heads_q, args.cache.dim)
    if workspace is None:
        workspace = make_tree_workspace(args, stream)
    ws_bytes = _workspace_bytes(workspace)
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
        out_status = _empty(stream, args.B, dtype=torch.int32, like=workspace.device)
    else:
        _check_out("out_status", out_status, (args.B,), torch.int32)
    rc = lib.spec_tree_attention(ctypes.byref(args), _ptr(out), out.stride(0), out.stride(1), _ptr(out_lse),
                                 _ptr(out_status), _ptr(workspace), ws_bytes, _stream_handle(stream))
    _raise(rc, "spec_tree_attention")
    return out, out_lse, out_status


# ------------------------------------------------------- attention weights

def make_weigh_args(*, q, lse, cu_rows, max_rows: int, cache: SpecCache, block_table, kv_len, scale=None,
                    layer: int = 0) -> SpecWeighArgs:
    """``spec_weigh_args``: q [rows, heads_q, dim] and lse [rows, heads_q] of
    the last rows of each request's cache, kv_len [B]."""
    _check_vectors("q", q, 3, cache.torch_dtype)
    _check_shape("q", q, (q.shape[0], q.shape[1], cache.dim))
    _check_f32("lse", lse)
    _check_shape("lse", lse, q.shape[:2])
    _check_i32("cu_rows", cu_rows)
    B = cu_rows.numel() - 1
    _check_table("block_table", block_table, B)
    _check_lengths("kv_len", kv_len, B)
    a = SpecWeighArgs()
    a.B, a.total_rows, a.max_rows, a.heads_q = B, q.shape[0], _int32("max_rows", max_rows), q.shape[1]
    a.layer = _int32("layer", layer)
    a.scale = cache.dim ** -0.5 if scale is None else float(scale)
    a.cu_rows, a.q, a.lse = _ptr(cu_rows), _ptr(q), _ptr(lse)
    a.sq_row, a.sq_head = q.stride()[:2]
    a.cache = cache
    a.block_table, a.ld_table, a.kv_len = _ptr(block_table), block_table.shape[1], _ptr(kv_len)
    a._keep = (q, lse, cu_rows, cache, block_table, kv_len)
    return a


def spec_attention_weights(args: SpecWeighArgs, before=None, *, ld=None, out=None, out_status=None, stream=None):
    """The cached keys' accumulated attention weights through
    ``spec_attention_weights``: `before` [B, heads, ld] float32 (None: zero)
    and what these rows add.  Returns (weights [B, heads, ld] float32, status
    [B] int32).  `out` may be `before`; `ld` is needed only without both."""
    import torch

    lib = _lib()
    given = before if before is not None else out
    ld = given.shape[-1] if given is not None else ld
    if ld is None:
        raise ValueError("the row length ld is needed where neither before nor out is given")
    shape = (args.B, args.cache.heads, _int32("ld", ld))
    _check_out("before", before, shape, torch.float32)
    _check_out("out", out, shape, torch.float32)
    _check_out("out_status", out_status, (args.B,), torch.int32)
    if out is None:
        out = _empty(stream, *shape, dtype=torch.float32, like=_device())
    if out_status is None:
        out_status = _empty(stream, args.B, dtype=torch.int32, like=_device())
    # the block stays as it is: another thread may call with it and another ld
    call = SpecWeighArgs.from_buffer_copy(args)
    call.ld = shape[2]
    rc = lib.spec_attention_weights(ctypes.byref(call), _ptr(before), _ptr(out), _ptr(out_status),
                                    _stream_handle(stream))
    _raise(rc, "spec_attention_weights")
    return out, out_status


# ---------------------------------------------------- eviction, commitment

def make_evict_args(*, weights, kv_len, keep: int, cache: SpecCache, block_table, to_table, sink: int = 0,
                    recent: int = 0, layer: int = 0) -> SpecEvictArgs:
    """``spec_evict_args``: weights [B, heads, ld] float32, kv_len [B],
    block_table [B, pages] and to_table [B, pages] (the new pages)."""
    _check_f32("weights", weights)
    _check_i32("kv_len", kv_len)
    B = kv_len.numel()
    if weights.dim() != 3 or tuple(weights.shape[:2]) != (B, cache.heads):
        raise ValueError(f"weights must have shape ({B}, {cache.heads}, ld), got {tuple(weights.shape)}")
    _check_table("block_table", block_table, B)
    _check_table("to_table", to_table, B)
    a = SpecEvictArgs()
    a.B, a.keep, a.ld = B, _int32("keep", keep), weights.shape[2]
    a.sink, a.recent, a.layer = _int32("sink", sink), _int32("recent", recent), _int32("layer", layer)
    a.weights, a.kv_len, a.cache = _ptr(weights), _ptr(kv_len), cache
    a.block_table, a.ld_table = _ptr(block_table), block_table.shape[1]
    a.to_table, a.ld_to = _ptr(to_table), to_table.shape[1]
    a._keep = (weights, kv_len, cache, block_table, to_table)
    return a


def spec_cache_evict(args: SpecEvictArgs, *, out_index=None, out_kept=None, out_len=None, out_status=None,
                     stream=None):
    """Keeps the tokens of largest weight through ``spec_cache_evict`` and
    moves them to the new pages.  Returns (index [B, heads, keep] int32, kept
    weights [B, heads, keep] float32, new lengths [B] int32, status [B]).
    `out_len` may be the block's kv_len."""
    import torch

    lib = _lib()
    shape = (args.B, args.cache.heads, args.keep)
    got = []
    for name, t, sh, dt in (("out_index", out_index, shape, torch.int32), ("out_kept", out_kept, shape, torch.float32),
                            ("out_len", out_len, shape[:1], torch.int32),
                            ("out_status", out_status, shape[:1], torch.int32)):
        _check_out(name, t, sh, dt)
        got.append(_empty(stream, *sh, dtype=dt, like=_device()) if t is None else t)
    index, kept, new_len, status = got
    rc = lib.spec_cache_evict(ctypes.byref(args), _ptr(index), _ptr(kept), _ptr(new_len), _ptr(status),
                              _stream_handle(stream))
    _raise(rc, "spec_cache_evict")
    return index, kept, new_len, status


def make_commit_args(*, k_new, v_new, cu_nodes, path, path_len, cache: SpecCache, block_table,
                     ctx_len) -> SpecCommitArgs:
    """``spec_commit_args``: k_new and v_new [layers, nodes, heads, dim] (or
    [nodes, heads, dim] for a cache of one layer), path [B, length] int32
    nodes of each request, path_len [B]."""
    if k_new.dim() == 3:
        k_new, v_new = k_new[None], v_new[None]
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _check_vectors(name, t, 4, cache.torch_dtype)
        _check_shape(name, t, (cache.layers, k_new.shape[1], cache.heads, cache.dim))
    if k_new.numel() > 0 and k_new.stride() != v_new.stride():
        raise ValueError("k_new and v_new must have the same strides")
    _check_i32("cu_nodes", cu_nodes)
    B = cu_nodes.numel() - 1
    _check_table("path", path, B)
    _check_lengths("path_len", path_len, B)
    _check_table("block_table", block_table, B)
    _check_lengths("ctx_len", ctx_len, B)
    a = SpecCommitArgs()
    a.B, a.total_nodes, a.cu_nodes = B, k_new.shape[1], _ptr(cu_nodes)
    a.k_new, a.v_new = _ptr(k_new), _ptr(v_new)
    a.sn_layer, a.sn_node, a.sn_head = k_new.stride()[:3]
    a.path, a.path_len, a.cache = _ptr(path), _ptr(path_len), cache
    a.block_table, a.ctx_len = _ptr(block_table), _ptr(ctx_len)
    a.ld_path, a.ld_table = path.shape[1], block_table.shape[1]
    a._keep = (k_new, v_new, cu_nodes, path, path_len, cache, block_table, ctx_len)
    return a


def spec_cache_commit(args: SpecCommitArgs, *, out_len=None, out_status=None, stream=None):
    """Writes the accepted paths' keys and values to the cache through
    ``spec_cache_commit``.  Returns (new lengths [B] int32, status [B]).
    `out_len` may be the block's ctx_len."""
    import torch

    lib = _lib()
    got = []
    for name, t in (("out_len", out_len), ("out_status", out_status)):
        _check_out(name, t, (args.B,), torch.int32)
        got.append(_empty(stream, args.B, dtype=torch.int32, like=_device()) if t is None else t)
    rc = lib.spec_cache_commit(ctypes.byref(args), _ptr(got[0]), _ptr(got[1]), _stream_handle(stream))
    _raise(rc, "spec_cache_commit")
    return got[0], got[1]


# ------------------------------------------------------------------- beams

def make_beam_args(*, logits, V: int, scores, keep: int, finished=None, end_token: int = 0) -> SpecBeamArgs:
    """``spec_beam_args``: logits [B*W, ld] (bf16 or fp32), scores [B, W]
    float32, finished [B, W] int32 (None: no beam has ended)."""
    _check_f32("scores", scores)
    if scores.dim() != 2:
        raise ValueError(f"scores must have shape (B, W), got {tuple(scores.shape)}")
    B, W = scores.shape
    if logits.dim() != 2 or logits.stride(1) != 1 or not logits.is_cuda:
        raise TypeError("logits must be a 2-D CUDA tensor with unit inner stride")
    if logits.shape[0] != B * W or logits.shape[1] < V:
        raise ValueError(f"logits must have {B * W} rows of at least {V}, got {tuple(logits.shape)}")
    if finished is not None:
        _check_i32("finished", finished)
        _check_shape("finished", finished, (B, W))
    a = SpecBeamArgs()
    a.B, a.W, a.keep, a.V, a.dtype = B, W, _int32("keep", keep), _int32("V", V), _dtype_code(logits)
    a.end_token = _int32("end_token", end_token)
    a.logits, a.ld = _ptr(logits), logits.stride(0)
    a.scores, a.finished = _ptr(scores), _ptr(finished)
    a._keep = (logits, scores, finished)
    return a


def spec_beam_workspace_bytes(args: SpecBeamArgs) -> int:
    return int(_lib().spec_beam_workspace_bytes(ctypes.byref(args)))


def make_beam_workspace(args: SpecBeamArgs, stream=None):
    import torch

    return _empty(stream, max(spec_beam_workspace_bytes(args), 256), dtype=torch.uint8, like=_device())


def spec_beam_select(args: SpecBeamArgs, *, workspace=None, out_scores=None, out_parents=None, out_tokens=None,
                     out_status=None, stream=None):
    """The best continuations over beams and vocabulary through
    ``spec_beam_select``.  Returns (scores [B, keep] float32, parents [B,
    keep] int32, tokens [B, keep] int32, status [B] int32)."""
    import torch

    lib = _lib()
    if workspace is None:
        workspace = make_beam_workspace(args, stream)
    ws_bytes = _workspace_bytes(workspace)
    shape = (args.B, args.keep)
    got = []
    for name, t, sh, dt in (("out_scores", out_scores, shape, torch.float32),
                            ("out_parents", out_parents, shape, torch.int32),
                            ("out_tokens", out_tokens, shape, torch.int32),
                            ("out_status", out_status, shape[:1], torch.int32)):
        _check_out(name, t, sh, dt)
        got.append(_empty(stream, *sh, dtype=dt, like=workspace.device) if t is None else t)
    rc = lib.spec_beam_select(ctypes.byref(args), *(_ptr(t) for t in got), _ptr(workspace), ws_bytes,
                              _stream_handle(stream))
    _raise(rc, "spec_beam_select")
    return tuple(got)


def _state(src, dst, B, W, keep, layered):
    """``spec_beam_state`` of src [B, W, ...] or [outer, B, W, ...]."""
    for name, t in (("a state's source", src), ("a state's destination", dst)):
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
    if src.dtype != dst.dtype or src.dim() != dst.dim():
        raise TypeError("a state's source and destination must have the same type and number of axes")
    fits = [tuple(src.shape[i:i + 2]) == (B, W) and tuple(dst.shape[i:i + 2]) == (B, keep)
            and src.shape[:i] == dst.shape[:i] and src.shape[i + 2:] == dst.shape[i + 2:] for i in (0, 1)]
    if layered is not None:
        fits[not layered] = False
    if all(fits):
        raise ValueError(f"a state of shape {tuple(src.shape)} may or may not have an axis before the request's: "
                         f"say which by `layered`")
    if not any(fits):
        raise ValueError(f"a state must have shapes (..., {B}, {W}, ...) and (..., {B}, {keep}, ...) with "
                         f"{'at most one' if layered is None else 'one' if layered else 'no'} axis before the "
                         f"request's, got {tuple(src.shape)} and {tuple(dst.shape)}")
    lead = int(fits[1])
    rest = 1
    for n, s, d in zip(reversed(src.shape[lead + 2:]), reversed(src.stride()[lead + 2:]),
                       reversed(dst.stride()[lead + 2:])):
        if n != 1 and (s != rest or d != rest):
            raise ValueError("the axes after a state's beams must be contiguous")
        rest *= n
    es = src.element_size()
    a = SpecBeamState()
    a.src, a.dst, a.row_bytes, a.outer = _ptr(src), _ptr(dst), rest * es, src.shape[0] if lead else 1
    a.src_outer, a.dst_outer = (src.stride(0) * es, dst.stride(0) * es) if lead else (0, 0)
    a.src_batch, a.src_beam = src.stride(lead) * es, src.stride(lead + 1) * es
    a.dst_batch, a.dst_beam = dst.stride(lead) * es, dst.stride(lead + 1) * es
    return a


def make_reorder_args(*, parents, beams: int, states, layered=None) -> ReorderArgs:
    """The arguments of ``spec_beam_reorder``: parents [B, keep] int32 and
    pairs (source [B, beams, ...], destination [B, keep, ...]), or both with
    one axis (layers) before the request's.  `layered` says whether states
    have that axis: True, False, a sequence of these for each state, or None,
    where shapes tell; a shape that fits both forms is refused then."""
    _check_i32("parents", parents)
    if parents.dim() != 2:
        raise ValueError(f"parents must have shape (B, keep), got {tuple(parents.shape)}")
    B, keep = parents.shape
    W = _int32("beams", beams)
    states = list(states)
    forms = [layered] * len(states) if layered is None or isinstance(layered, bool) else list(layered)
    if len(forms) != len(states):
        raise ValueError(f"layered must have one value for each of {len(states)} states, got {len(forms)}")
    block = (SpecBeamState * max(1, len(states)))(*(_state(s, d, B, W, keep, f)
                                                    for (s, d), f in zip(states, forms)))
    return ReorderArgs(B, W, keep, parents, (block, len(states)), (parents, states))


def spec_beam_reorder(args: ReorderArgs, *, stream=None):
    """The beams' states in their new order through ``spec_beam_reorder``:
    dst[..., b, j] = src[..., b, parents[b, j]], zero where the parent is
    outside the beams.  Returns nothing."""
    block, n = args.states
    rc = _lib().spec_beam_reorder(args.B, args.W, args.keep, args.parents, block, n, _stream_handle(stream))
    _raise(rc, "spec_beam_reorder")
