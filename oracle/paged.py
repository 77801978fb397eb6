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
