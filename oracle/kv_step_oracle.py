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
