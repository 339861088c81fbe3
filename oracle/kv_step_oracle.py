"""CPU oracle of a step's tables and of the rotated append to the 4-bit key/value cache.

Test infrastructure only, written from the definitions with numpy and Python integers.  The
roundings to float32 are part of the rotation's definition.
"""
from __future__ import annotations

import numpy as np

from oracle import kv_oracle as kv


def tables(page, kv_len, count, free, taken, table, rows):
    """(table, kv_len, row_start, taken, position, slot) of a step, sequence by sequence."""
    table = np.array(table, np.int64)
    batch, most = table.shape
    new_len, row_start = [], [0]
    position, slot = np.full(rows, -1, np.int64), np.full(rows, -1, np.int64)
    taken = max(0, int(taken))
    for b in range(batch):
        length = min(max(int(kv_len[b]), 0), most * page)
        n = min(max(int(count[b]), 0), most * page - length)
        for p in range(length, length + n):
            if p % page == 0:   # a new page begins
                table[b, p // page] = free[taken] if taken < len(free) else -1
                taken += 1
            r = row_start[-1] + p - length
            if r < rows:
                position[r] = p
                if table[b, p // page] >= 0:
                    slot[r] = table[b, p // page] * page + p % page
        new_len.append(length + n)
        row_start.append(row_start[-1] + n)
    return table, np.array(new_len), np.array(row_start), taken, position, slot


def turned(x, weight, cos_sin, positions, eps=1e-6, interleaved=False):
    """Rows x [n, heads, D] normalised (with a weight) and rotated, in float32; NaN where cos_sin has no such position."""
    x = np.array(x, np.float32)
    with np.errstate(all="ignore"):
        if weight is not None:
            wide = x.astype(np.float64)
            u = (1.0 / np.sqrt((wide * wide).sum(-1, keepdims=True) / x.shape[-1] + eps)).astype(np.float32)
            x = (x * u) * np.asarray(weight, np.float32)
        if cos_sin is None:
            return x
        half = cos_sin.shape[-1]
        known = (positions >= 0) & (positions < len(cos_sin))
        cs = cos_sin[np.where(known, positions, 0)][:, None]
        i = np.arange(half)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y = x.copy()
        y[..., a] = x[..., a] * cs[:, :, 0] - x[..., b] * cs[:, :, 1]
        y[..., b] = x[..., b] * cs[:, :, 0] + x[..., a] * cs[:, :, 1]
        y[(positions >= len(cos_sin))] = np.nan
    return y


def row_positions(rows, row_start, kv_len, table, page):
    """Position of each row; None-like -(1 << 40) where it belongs to no sequence."""
    at = np.full(rows, -(1 << 40), np.int64)
    for r0, n, length in kv.sequences(rows, len(kv_len), row_start, kv_len, table, page):
        at[r0:r0 + n] = length - n + np.arange(n)
    return at


def append_rotated(cache, q, k, v, row_start, kv_len, table, cos_sin, q_weight=None, k_weight=None, eps=1e-6,
                   interleaved=False, fill=0.0):
    """Writes the cache; the rotated queries in float32 (`fill` in rows that belong to no sequence)."""
    at = row_positions(len(q), row_start, kv_len, table, cache.page)
    out = turned(q, q_weight, cos_sin, at, eps, interleaved)
    out[at < 0] = 0.0
    out[at == -(1 << 40)] = fill
    with np.errstate(all="ignore"):
        kv.append(cache, turned(k, k_weight, cos_sin, at, eps, interleaved), np.asarray(v, np.float32), row_start, kv_len, table)
    return out


def sees(position, t, causal, window, sinks):
    """Which of the positions t a row at `position` sees."""
    see = np.ones(len(t), bool)
    if causal:
        see &= t <= position
    if window:
        see &= (t > position - window) | (t < sinks)
    return see


def attention(cache, q, row_start, kv_len, table, scale=None, causal=True, window=0, sinks=0, prefix=None, fill=0.0, spread=None):
    """kv_oracle.attention with sinks and with a prefix = (table [pages], length) that holds the first positions
    of every sequence: (O, lse, A, E) in float64."""
    rows, q_heads, dim = q.shape
    per, page = q_heads // cache.heads, cache.page
    scale = dim ** -0.5 if scale is None else scale
    o, a = np.full(q.shape, fill, np.float64), np.zeros(q.shape, np.float64)
    lse, err = np.full(q.shape[:2], fill, np.float64), np.zeros(q.shape[:2], np.float64)
    common = min(max(int(prefix[1]), 0), len(prefix[0]) * page) if prefix is not None else 0
    for b, (r0, n, length) in enumerate(kv.sequences(rows, len(kv_len), row_start, kv_len, table, page)):
        if n == 0:
            continue
        pg = [int(prefix[0][t // page] if t < common else table[b, t // page]) for t in range(length)]
        wanted = np.zeros(length, bool)
        for i in range(n):
            wanted |= sees(length - n + i, np.arange(length), causal, window, sinks)
        real = np.array([t for t in range(length) if wanted[t] and 0 <= pg[t] < len(cache.bytes)], int)
        got = [cache.read(pg[t], t % page) for t in real]
        kk, vv = (np.array([g[x] for g in got], np.float64).reshape(len(real), cache.heads, dim) for x in (0, 1))
        steps = np.zeros((len(real), cache.heads, dim))
        for x, t in enumerate(real):
            p = cache.pair_at(0, t % page)
            pair = np.ascontiguousarray(cache.bytes[pg[t]][:, p:p + 4 * (dim // cache.group)]).view(np.float16)
            steps[x] = np.repeat(pair.reshape(cache.heads, -1, 2)[..., 0].astype(np.float64), cache.group, -1)
        for i in range(n):
            see = sees(length - n + i, real, causal, window, sinks)
            for h in range(q_heads):
                if not see.any():
                    o[r0 + i, h], lse[r0 + i, h] = 0.0, -np.inf
                    continue
                with np.errstate(all="ignore"):
                    x = q[r0 + i, h].astype(np.float64)
                    s = kk[see, h // per] @ x * scale
                    top = s.max()
                    p = np.exp(s - top)
                    o[r0 + i, h] = p @ vv[see, h // per] / p.sum()
                    a[r0 + i, h] = p @ np.abs(vv[see, h // per]) / p.sum()
                    lse[r0 + i, h] = top + np.log(p.sum())
                    if spread is not None:
                        err[r0 + i, h] = scale * spread(steps[see, h // per], kk[see, h // per], x).max()
    return o, lse, a, err
