"""fp64 / integer oracle of the paged-cache operators: the maps of a step, rotary positions, rows
written to slots, and attention over pages (the pages gathered into one packed array, then the
cross-attention oracle). numpy; nothing here is shared with the library."""
from __future__ import annotations

import math

import numpy as np

from . import XProblem, xattn_fwd


def plan(ctx, new, free, table, page, num_pages, max_tokens):
    """(table, cu, lk, positions, slots, counts) of a step; see fat_paged_plan in fat_attn.h."""
    table = np.array(table, np.int64)
    n, width = table.shape
    pos, slots = np.zeros(max_tokens, np.int64), np.full(max_tokens, -1, np.int64)
    cu, lk, taken, t = [0], [], 0, 0
    for i in range(n):
        c, a = int(ctx[i]), int(new[i])
        if c < 0 or a < 0:
            c = a = 0
        fits = c + a <= width * page
        have, want = -(-c // page), -(-(c + a) // page)
        if fits:
            for col in range(have, want):
                p = int(free[taken]) if taken < len(free) else -1
                table[i, col] = p if 0 <= p < num_pages else -1
                taken += 1
        for j in range(a):
            if t < max_tokens:
                pos[t] = c + j
                if fits:
                    p = int(table[i, (c + j) // page])
                    slots[t] = p * page + (c + j) % page if 0 <= p < num_pages else -1
            t += 1
        cu.append(min(t, max_tokens))
        lk.append(c + a)
    return (table, np.array(cu), np.array(lk, np.int64), pos, slots, np.array([taken, t]))


def rope_angles(positions, rotary_dim, base=10000.0, factor=1.0, ramp=None):
    """[T, rotary_dim / 2] angles in radians (fp64, reduced with exact products below 2^53)."""
    out = np.zeros((len(positions), rotary_dim // 2))
    for i in range(rotary_dim // 2):
        theta = base ** (-2.0 * i / rotary_dim)
        if ramp is None:
            theta = theta / factor
        else:
            low, high, original = ramp
            keep = min(1.0, max(0.0, (original * theta / (2 * math.pi) - low) / (high - low)))
            theta = theta * (keep + (1.0 - keep) / factor)
        out[:, i] = np.asarray(positions, np.float64) * theta
    return out


def rope(x, positions, rotary_dim, base=10000.0, interleaved=True, factor=1.0, ramp=None,
         amplitude=1.0, inverse=False):
    """Rows x [T, H, d] (fp64) turned at positions; the transpose when inverse."""
    x = np.asarray(x, np.float64)
    a = rope_angles(positions, rotary_dim, base, factor, ramp)
    c, s = amplitude * np.cos(a)[:, None], amplitude * np.sin(a)[:, None]
    if inverse:
        s = -s
    y = x.copy()
    h = rotary_dim // 2
    first = np.arange(0, rotary_dim, 2) if interleaved else np.arange(h)
    second = first + (1 if interleaved else h)
    u, v = x[..., first], x[..., second]
    y[..., first] = u * c - v * s
    y[..., second] = u * s + v * c
    return y


def gather(cache, table, lk, num_pages):
    """Packed rows [sum lk, H, d] of a cache [pages, page, H, d] (pages outside: zeros)."""
    page = cache.shape[1]
    rows = [np.zeros((0,) + cache.shape[2:], cache.dtype)]
    for i, m in enumerate(lk):
        p = np.arange(int(m))
        pg = np.asarray(table, np.int64)[i, p // page]
        ok = (pg >= 0) & (pg < num_pages)
        row = np.zeros((len(p),) + cache.shape[2:], cache.dtype)
        row[ok] = cache[pg[ok], (p % page)[ok]]
        rows.append(row)
    return np.concatenate(rows)


def attention(q, k_cache, v_cache, block_table, cu_q, lk, **kw):
    """(out, lse, A, S, B) in fp64; kw as oracle.XProblem. The last three feed tolerances:
    A = sum_k P |V|, S = |scale| max sum_c |q_c k_c|, B = max |bias|."""
    k = gather(k_cache, block_table, lk, k_cache.shape[0])
    v = gather(v_cache, block_table, lk, v_cache.shape[0])
    cu_k = np.concatenate([[0], np.cumsum(lk)]).astype(np.int32)
    total = int(cu_q[-1])
    pb = dict(cu_seqlens_q=np.asarray(cu_q, np.int32), cu_seqlens_k=cu_k, **kw)
    out, lse = xattn_fwd(XProblem(q[:total], k, v, **pb))
    a, _ = xattn_fwd(XProblem(q[:total], k, np.abs(v), **pb))
    x = 0.0
    for i in range(len(lk)):
        group = q.shape[1] // k.shape[1]
        kq = np.abs(k[cu_k[i]:cu_k[i + 1]])
        qq = np.abs(q[cu_q[i]:cu_q[i + 1]])
        if len(kq) and len(qq):
            for h in range(q.shape[1]):
                x = max(x, float((qq[:, h] @ kq[:, h // group].T).max()))
    x *= abs(kw.get("scale", 1.0))
    b = 0.0
    if kw.get("table") is not None:
        b += float(np.abs(kw["table"]).max())
    if kw.get("slopes") is not None and len(lk):
        b += float(np.abs(kw["slopes"]).max()) * (int(max(lk)) + int(np.diff(cu_q).max()))
    return out, lse, a, x, b


def tree_plan(parents, cu_q, lk, total, max_nodes, words):
    """(positions [total], mask [total, words]) of trees of drafted tokens, node by node; bad parents count
    as -1, requests of more than max_nodes nodes or fewer keys than nodes get zeros."""
    pos, mask = np.zeros(total, np.int64), np.zeros((total, words), np.uint32)
    for i in range(len(lk)):
        sq, m = int(cu_q[i]), int(cu_q[i + 1] - cu_q[i])
        if m > max_nodes or lk[i] < m:
            continue
        paths = []
        for j in range(m):
            p = int(parents[sq + j])
            paths.append((paths[p] if 0 <= p < j else []) + [j])
            pos[sq + j] = int(lk[i]) - m + len(paths[j]) - 1
            for a in paths[j]:
                mask[sq + j, a // 32] |= np.uint32(1 << (a % 32))
    return pos, mask.view(np.int32)


def tree_attention(q, k_cache, v_cache, block_table, cu_q, lk, positions, mask, bias=None, bucket=None,
                   slopes=None, scale=1.0):
    """(out, lse, A, S, B) as of `attention`, for queries that see the context before their request's first
    one and the own keys of their mask bits. bucket(deltas): bucket of each key position - query position."""
    k, v = (gather(c, block_table, lk, k_cache.shape[0]) for c in (k_cache, v_cache))
    total, hq = int(cu_q[-1]), q.shape[1]
    group = hq // k.shape[1]
    out, lse = np.zeros((total, hq, q.shape[2])), np.full((hq, total), -np.inf)
    a, s, big, at = np.zeros_like(out), 0.0, 0.0, 0
    words = np.asarray(mask).view(np.uint32)
    for i in range(len(lk)):
        sq, m, n = int(cu_q[i]), int(cu_q[i + 1] - cu_q[i]), int(lk[i])
        ki, vi = k[at:at + n], v[at:at + n]
        at += n
        if m == 0 or n < m:
            continue
        c = n - m
        own = np.array([[(int(words[sq + j, b // 32]) >> (b % 32)) & 1 for b in range(m)]
                        for j in range(m)], bool)
        see = np.concatenate([np.ones((m, c), bool), own], 1)
        where = np.clip(np.asarray(positions[sq:sq + m], np.int64), c, n - 1)
        delta = np.concatenate([np.arange(c), where])[None] - where[:, None]
        for h in range(hq):
            qh, kh, vh = q[sq:sq + m, h], ki[:, h // group], vi[:, h // group]
            x, b = scale * (qh @ kh.T), np.zeros(delta.shape)
            s = max(s, abs(scale) * float((np.abs(qh) @ np.abs(kh).T).max()))
            if bias is not None:
                b = b + bias[bucket(delta), h]
            if slopes is not None:
                b = b - slopes[h] * np.abs(delta)
            big = max(big, float(np.abs(b).max()))
            x = np.where(see, x + b, -np.inf)
            top = x.max(1)
            some = np.isfinite(top)
            p = np.exp(x[some] - top[some, None])
            lse[h, sq:sq + m][some] = top[some] + np.log(p.sum(1))
            p /= p.sum(1, keepdims=True)
            out[sq:sq + m, h][some] = p @ vh
            a[sq:sq + m, h][some] = p @ np.abs(vh)
    return out, lse, a, s, big
