"""Plain 64-bit definitions of the operators beside the drafted tree, and the error bounds of their kernels (numpy)."""
from __future__ import annotations

import math

import numpy as np

from tree_ref import HALF, bits, cached, f64  # noqa: F401


# ---------------------------------------------------- norms and positions

def rotate(x, weight, positions, freq, eps, interleaved, dtype):
    """(y, its bound) of one side [rows, heads, dim].

    The mean of squares errs by dim roundings of positive terms, half of which a root keeps; 1 / sqrt, the products
    with it and the weight, and the turn's two products and sum add a rounding each (rsqrt two); sine and cosine err
    by 2^-23 and the angle by 2^-24 of a turn, 2 pi 2^-24 in size."""
    rows, heads, dim = x.shape
    rot = 2 * len(freq)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if weight is None else weight)
    a = np.outer(positions.astype(np.float64), freq.astype(np.float64))[:, None, :]
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out, size = y.copy(), np.abs(y)
    ya, yb = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = ya * np.cos(a) - yb * np.sin(a), yb * np.cos(a) + ya * np.sin(a)
    both = np.abs(ya) + np.abs(yb)
    size[..., ia], size[..., ib] = both, both
    f32 = HALF["fp32"]
    tol = size * ((dim / 2 + 8) * f32 + 2.0 ** -23 + 2 * math.pi * 2.0 ** -24) + np.abs(out) * HALF[dtype] + 2.0 ** -25
    return out, tol


# --------------------------------------------------------------- attention

def text(sees, ctx, window, sinks):
    """Which of the cached tokens and of the drafted ones a row sees: `sees` [n] says which drafted ones it would."""
    drafted = np.flatnonzero(sees)
    own = np.concatenate([np.arange(ctx), ctx + drafted])
    if window is not None and len(own) > window:
        last = own[len(own) - window:]
        own = np.union1d(own[:min(sinks, len(own))], last)
    out = np.zeros(ctx + len(sees), bool)
    out[own] = True
    return out


def e4m3(b):
    """The values of e4m3 bytes."""
    b = np.asarray(b, dtype=np.uint8).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >> 7, -v, v)


def nearest8(x):
    """e4m3 bytes of the values nearest to x (ties to even); infinities, NaN and what rounds past 448 are not asked."""
    table = e4m3(np.arange(127))
    a = np.abs(x)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - a, a - table[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def attention(q, k_new, v_new, cu, k, v, page, table, ctx, mask, scale, dtype, window=None, sinks=0, scales=None,
              block=None):
    """(out, lse, bound of out, bound of lse), all [nodes, heads_q, ...].

    k and v [pages, page, heads, dim]; with `scales` (of keys, of values, [pages, blocks, heads]) they are the bytes'
    values, and drafted ones have scale 1.  A score errs by the fp32 sum over dim channels and by the products with
    the scales; an exponential by 2^-21 and the rounding of its argument; sums over keys add a rounding a key.  Weights
    are rounded to the cache's type, or with 8 bits to fp16: half a step of 2^-24, 2^-31 of the largest weight, which
    is 2^6 or more, at least."""
    total, hq, dim = q.shape
    heads = k_new.shape[1]
    group = hq // heads
    out, lse = np.zeros((total, hq, dim)), np.full((total, hq), -np.inf)
    out_tol, lse_tol = np.zeros((total, hq, dim)), np.zeros((total, hq))
    half, f32 = HALF[dtype], HALF["fp32"]
    for b in range(len(ctx)):
        n, c = cu[b + 1] - cu[b], int(ctx[b])
        if n <= 0:
            continue
        tree = np.stack([(np.arange(n) <= i) if mask is None else bits(mask[cu[b] + i], n) for i in range(n)])
        sees = np.stack([text(t, c, window, sinks) for t in tree])
        for g in range(heads):
            kk = np.concatenate([cached(k, table[b], page, c, g), k_new[cu[b]:cu[b + 1], g]])
            vv = np.concatenate([cached(v, table[b], page, c, g), v_new[cu[b]:cu[b + 1], g]])
            vs = np.ones(c + n)
            if scales is not None:
                pos = np.arange(c)
                at = (table[b][pos // page], pos % page // block, g)
                kk[:c] *= scales[0][at][:, None]
                vv[:c] *= scales[1][at][:, None]
                vs[:c] = scales[1][at]
            for h in range(g * group, (g + 1) * group):
                for i in range(n):
                    row, see = cu[b] + i, sees[i]
                    if not see.any():
                        continue
                    s = kk[see] @ q[row, h] * scale
                    m = s.max()
                    e = np.exp(s - m)
                    lse[row, h] = m + math.log(e.sum())
                    p = e / e.sum()
                    with np.errstate(invalid="ignore"):
                        out[row, h] = p @ vv[see]
                        away = p @ np.abs(vv[see])
                    size = (np.abs(kk[see]) @ np.abs(q[row, h])).max() * abs(scale)
                    ns = see.sum()
                    ds = (dim + 8) * f32 * size + 2.0 ** -21
                    if scales is None:
                        out_tol[row, h] = away * (half + 2 * ds + 2 * (ns + 16) * f32) + np.abs(out[row, h]) * half + 1e-30
                    else:
                        lv = np.abs(np.log2(np.maximum(vs[see], 2.0 ** -60))).max()
                        ds += (4 * size + 2 * lv + 32) * f32
                        top = (p * vs[see]).max()
                        small = 2.0 ** -31 * top * (np.abs(vv[see]) / np.maximum(vs[see], 2.0 ** -60)[:, None]).sum(0)
                        out_tol[row, h] = (away * (2.0 ** -11 + 2 * ds + 2 * (ns + 16) * f32) + small +
                                           np.abs(out[row, h]) * half + 2.0 ** -50 + (2.0 ** -25 if dtype == "fp16" else 0))
                    lse_tol[row, h] = ds + (ns + 16) * f32 + 4 * f32 * abs(lse[row, h])
    return out, lse, out_tol, lse_tol


# -------------------------------------------------------------- commitment

def scale_for(top):
    """The smallest power of two from 2^-126 on whose 448-fold reaches top (0 for 0)."""
    if top == 0:
        return 0.0
    k = -126
    while 448.0 * 2.0 ** k < top:
        k += 1
    return 2.0 ** k


def commit8(held, scale, x, cu, path, path_len, table, ctx, page, block):
    """One side of the cache after commitment: bytes [layers, pages, page, heads, dim] and scales [layers, pages,
    blocks, heads], of x [layers, nodes, heads, dim] float64.  The rounding is of the product that the definition
    names, in fp32."""
    held, scale = held.copy(), scale.copy()
    layers, _, _, heads, dim = held.shape
    for b in range(len(ctx)):
        a, m = int(ctx[b]), int(path_len[b])
        for j in range(a // block, (a + m - 1) // block + 1 if m else a // block):
            lo, hi = max(a, j * block), min(a + m, (j + 1) * block)
            p, s0 = table[b, j * block // page], j * block % page
            new = x[:, cu[b] + path[b, lo - a:hi - a]]
            for l in range(layers):
                for h in range(heads):
                    part = new[l, :, h]
                    fine = np.isfinite(part)
                    need = np.float32(scale_for(np.abs(part[fine]).max() if fine.any() else 0.0))
                    old = np.float32(scale[l, p, s0 // block, h])
                    before = j * block < a
                    s = need if not before or need > old else old
                    inv = np.float32(0) if s == 0 else np.float32(1) / s
                    if before and need > old:
                        rows = slice(s0, s0 + a - j * block)
                        was = e4m3(held[l, p, rows, h]).astype(np.float32)
                        again = nearest8(((was * old) * inv).astype(np.float64))
                        held[l, p, rows, h] = np.where(np.isnan(was), 0x7f, again)
                    scale[l, p, s0 // block, h] = s
                    y = np.where(fine, part, 0.0).astype(np.float32) * inv
                    held[l, p, s0 + lo - j * block:s0 + hi - j * block, h] = np.where(fine, nearest8(y.astype(np.float64)), 0x7f)
    return held, scale
