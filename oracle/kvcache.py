"""Oracle: the paged key-value-cache calls, written from their definitions in fp64.

TEST INFRASTRUCTURE ONLY, as the rest of this package: NumPy loops over the
definitions in include/fkmeans.h, sharing nothing with the HIP path. The pages
name KV-cache compression and attention routing only as uses of the clusters
("flash-kmeans and the return of exact K-Means on the GPU", introduction);
they give no values for them, so parity is pinned by the definitions.
"""
from __future__ import annotations

import numpy as np


def page_tables(len_old, len_new, table_in, free_pages, page, width, tokens):
    """Request by request, page by page: the six outputs as int64 arrays."""
    B = len(len_old)
    table = np.full((B, width), -1, np.int64)
    slots, positions = np.full(tokens, -1, np.int64), np.zeros(tokens, np.int64)
    cu_tokens, cu_pages = np.zeros(B + 1, np.int64), np.zeros(B + 1, np.int64)
    lens = np.zeros(B, np.int64)
    t = f = 0
    for b in range(B):
        old, new = max(int(len_old[b]), 0), max(int(len_new[b]), 0)
        lens[b] = old + new
        for j in range(width):
            if j * page >= old + new:
                break
            if j * page < old:                       # a page the request has
                if table_in is not None and j < table_in.shape[1]:
                    table[b, j] = table_in[b, j]
            else:
                if f < len(free_pages):
                    table[b, j] = free_pages[f]
                f += 1
        for i in range(new):
            if t < tokens:
                p = old + i
                positions[t] = p
                if p // page < width and table[b, p // page] >= 0:
                    slots[t] = table[b, p // page] * page + p % page
            t += 1
        cu_tokens[b + 1], cu_pages[b + 1] = t, f
    return table, lens, cu_tokens, cu_pages, slots, positions


def norm_rope(x, weight, eps, rope, positions, interleaved):
    """x (T,H,D) float64 -> (y, m): the result, and for each element the sum of
    the magnitudes of the terms it is a sum of (the scale of its rounding)."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    m = np.abs(y)
    if rope is None or rope.shape[1] == 0:
        return y, m
    rot = rope.shape[1]
    half = rot // 2
    p = np.clip(positions, 0, rope.shape[0] - 1)
    out, mag = y.copy(), m.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = rope[p, i][:, None], rope[p, half + i][:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        mag[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
        mag[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
    return out, mag


def paged_attn(q, k_cache, v_cache, table, lens, scale, softcap=0.0, bias=None):
    """q (B,Hq,D), caches (pages,page,Hkv,D) float64 -> (out, lse, info).
    info[b,h] = (largest |s|, largest sum |q_i k_i| scale, largest |v|, keys)
    over the keys that count, for error bounds."""
    B, Hq, D = q.shape
    pages, page, Hkv, _ = k_cache.shape
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    info = np.zeros((B, Hq, 4))
    for b in range(B):
        n = min(int(lens[b]), table.shape[1] * page)
        at = [(int(table[b, j // page]), j % page) for j in range(n)]
        at = [(p, t) for p, t in at if 0 <= p < pages]
        if not at:
            continue
        pi, ti = np.array(at).T
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            keep = np.ones(len(pi), bool)
            if bias is not None:
                keep = bias[pi, ti, hk] != -np.inf
            p, t = pi[keep], ti[keep]
            if not len(p):
                continue
            k, v = k_cache[p, t, hk], v_cache[p, t, hk]
            raw = scale * (k @ q[b, h])
            s = softcap * np.tanh(raw / softcap) if softcap > 0 else raw
            if bias is not None:
                s = s + bias[p, t, hk]
            top = s.max()
            w = np.exp(s - top)
            lse[b, h] = top + np.log(w.sum())
            out[b, h] = (w / w.sum()) @ v
            info[b, h] = (np.abs(raw).max(), abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max(),
                          np.abs(v).max(), len(p))
    return out, lse, info


def prompt_attn(q, k_cache, v_cache, table, lens, cu, scale, softcap=0.0, bias=None):
    """q (T,Hq,D): token cu[b] + i of request b over its keys up to place
    lens[b] - n + i, n = cu[b+1] - cu[b]. -> (out, lse, info) as paged_attn, NaN in
    rows of tokens that no request has."""
    T, Hq, D = q.shape
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    info = np.zeros((T, Hq, 4))
    for b in range(len(lens)):
        n = int(cu[b + 1]) - int(cu[b])
        for i in range(n):
            t = int(cu[b]) + i
            seen = max(int(lens[b]) - n + i + 1, 0)
            o, s, f = paged_attn(q[t:t + 1], k_cache, v_cache, table[b:b + 1], [seen], scale, softcap, bias)
            out[t], lse[t], info[t] = o[0], s[0], f[0]
    return out, lse, info


def e4m3_round(y):
    """Nearest e4m3 number (multiples of 2^-9 up to 2^-6, then eight to a binade, up to 448), ties
    to the even multiple; |y| <= 448."""
    a = np.abs(y)
    _, e = np.frexp(np.maximum(a, 2.0 ** -6))            # a = f 2^e, 0.5 <= f < 1
    step = np.ldexp(1.0, e - 4)
    return np.sign(y) * np.rint(a / step) * step


def quantise(x):
    """Rows x (..., D) float64 -> (numbers that the codes stand for, scale (...)): the scale
    is the smallest power of two >= 2^-126 that takes the largest finite element to 448
    at most (1 for zeros); what is not finite is NaN."""
    ok = np.isfinite(x)
    most = np.where(ok, np.abs(x), 0.0).max(-1)
    scale = np.ones(most.shape)
    for at in np.ndindex(most.shape):
        if most[at] > 0:
            s = 2.0 ** -126
            while 448 * s < most[at]:
                s *= 2
            scale[at] = s
    y = np.where(ok, x, 0.0) / scale[..., None]
    return np.where(ok, e4m3_round(y) * scale[..., None], np.nan), scale
