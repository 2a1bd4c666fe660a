"""Plain 64-bit implementations of the drafted-tree operators and the error
bounds of their kernels, for the GPU tests (numpy, one request at a time)."""
from __future__ import annotations

import math

import numpy as np

#: half a step of a rounding, relative to the value
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def f64(t):
    return t.detach().double().cpu().numpy()


def cached(cache, table_row, page, length, head):
    """The first `length` tokens of a request: cache [pages, page, heads, dim] as float64."""
    pos = np.arange(length)
    return cache[table_row[pos // page], pos % page, head]


def bits(mask_row, n):
    return np.array([bool((int(mask_row[j // 32]) >> (j % 32)) & 1) for j in range(n)], dtype=bool)


def attention(q, k_new, v_new, cu, k, v, page, table, ctx, mask, scale, dtype):
    """(out, lse, bound of out, bound of lse), all [nodes, heads_q, ...].

    The kernel's scores err by the fp32 sum over dim channels (dim + 4
    roundings of terms of size |q||k|) and its exponentials by 2^-21; a weight
    is rounded once to the cache's type, sums over keys add one fp32 rounding
    a key, and the result is rounded once more."""
    total, hq, dim = q.shape
    heads = k_new.shape[1]
    group = hq // heads
    out, lse = np.zeros((total, hq, dim)), np.full((total, hq), -np.inf)
    out_tol, lse_tol = np.zeros((total, hq, dim)), np.zeros((total, hq))
    half, f32 = HALF[dtype], HALF["fp32"]
    for b in range(len(ctx)):
        n, c = cu[b + 1] - cu[b], int(ctx[b])
        for h in range(hq):
            g = h // group
            kk = np.concatenate([cached(k, table[b], page, c, g), k_new[cu[b]:cu[b + 1], g]])
            vv = np.concatenate([cached(v, table[b], page, c, g), v_new[cu[b]:cu[b + 1], g]])
            for i in range(n):
                row = cu[b] + i
                see = np.concatenate([np.ones(c, bool), (np.arange(n) <= i) if mask is None else bits(mask[row], n)])
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
                # |s| again: its product with the scale and log2(e), each rounded
                ds = (dim + 8) * f32 * size + 2.0 ** -21
                ns = see.sum()
                out_tol[row, h] = away * (half + 2 * ds + 2 * (ns + 16) * f32) + np.abs(out[row, h]) * half + 1e-30
                lse_tol[row, h] = ds + (ns + 16) * f32 + 4 * f32 * abs(lse[row, h])
    return out, lse, out_tol, lse_tol


def weights(q, lse, cu, k, page, table, length, scale, before, ld):
    """(weights, their bound) [B, heads, ld]."""
    hq, heads = q.shape[1], k.shape[2]
    group, dim = hq // heads, q.shape[2]
    B = len(length)
    out, tol = np.zeros((B, heads, ld)), np.zeros((B, heads, ld))
    f32 = HALF["fp32"]
    for b in range(B):
        n, a = cu[b + 1] - cu[b], int(length[b])
        for g in range(heads):
            kk = cached(k, table[b], page, a, g)
            w, t = np.zeros(a), np.zeros(a)
            for i in range(n):
                see = np.arange(a) <= a - n + i
                for h in range(g * group, (g + 1) * group):
                    if np.isposinf(lse[cu[b] + i, h]):
                        continue
                    s = kk @ q[cu[b] + i, h] * scale
                    size = np.abs(kk) @ np.abs(q[cu[b] + i, h]) * abs(scale) + abs(lse[cu[b] + i, h])
                    p = np.where(see, np.exp(s - lse[cu[b] + i, h]), 0.0)
                    w += p
                    t += p * ((dim + 8) * f32 * size + 2.0 ** -21)
            old = 0.0 if before is None else before[b, g, :a]
            out[b, g, :a] = old + w
            tol[b, g, :a] = 2 * t + (n * group + 4) * f32 * (w + np.abs(old)) + 1e-30
    return out, tol


def evict(w, length, keep, sink, recent):
    """(index, kept weights) of one request and head."""
    m = min(length, keep)
    key = w[:length].astype(np.float64).copy()
    nan = np.isnan(key)
    rank = np.lexsort((np.arange(length), -np.where(nan, 0.0, key), nan))  # NaN last, then the largest, then the first
    always = [j for j in range(length) if j < sink or j >= length - recent]
    if length <= keep:
        chosen = np.arange(length)
    else:
        rest = [j for j in rank if sink <= j < length - recent]
        chosen = np.sort(np.array(always + rest[:keep - len(always)], dtype=np.int64))
    index, kept = np.full(keep, -1, np.int32), np.zeros(keep, np.float32)
    index[:m], kept[:m] = chosen, w[chosen]
    return index, kept


def beams(z, cum, ended, end_token, keep):
    """(scores, parents, tokens, gaps) of one request: z [W, V], cum [W].  A
    gap is the distance to the next candidate; -1 tokens where there is none."""
    W, V = z.shape
    total = np.full((W, V), -np.inf)
    for w in range(W):
        if cum[w] == -np.inf:
            continue
        if ended is not None and ended[w]:
            total[w, end_token] = cum[w]
        else:
            m = z[w].max()
            if m > -np.inf:
                total[w] = cum[w] + (z[w] - (m + math.log(np.exp(z[w] - m).sum())))
    flat = total.ravel()
    order = np.lexsort((np.arange(W * V), -flat))[:keep + 1]
    val = flat[order]
    scores, parents, tokens = np.full(keep, -np.inf), np.full(keep, -1, np.int32), np.full(keep, -1, np.int32)
    gaps = np.full(keep, np.inf)
    for i in range(min(keep, W * V)):
        if val[i] > -np.inf:
            scores[i], parents[i], tokens[i] = val[i], order[i] // V, order[i] % V
            if i + 1 < len(val):
                gaps[i] = val[i] - val[i + 1]
    return scores, parents, tokens, gaps
