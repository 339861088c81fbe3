"""CPU oracle of the 4-bit key/value cache: quantiser, byte layout, attention.

Test infrastructure only, written from the definitions with numpy.  The
quantiser is float32 (its roundings are part of the definition); attention is
float64.
"""
from __future__ import annotations

import numpy as np

NIBBLE_ORDER = (0, 2, 4, 6, 1, 3, 5, 7)
MAX_ABS = np.float32(32768.0)


def quantise(x, group):
    """x [..., D] -> codes uint8 [..., D], step and lowest value float16 [..., D/group]."""
    x = np.asarray(x, np.float32)
    xs = x.reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        lo = xs.min(-1).astype(np.float16)
        lof = lo.astype(np.float32)
        step = (np.maximum(xs.max(-1) - lof, np.float32(0)) * (np.float32(1) / np.float32(15))).astype(np.float16)
        sf = step.astype(np.float32)
        q = np.rint((xs - lof[..., None]) / sf[..., None])
        q = np.where(sf[..., None] > 0, np.clip(np.nan_to_num(q, nan=0.0), 0, 15), 0)
    return q.astype(np.uint8).reshape(x.shape), step, lo


def quantise_token(k, v, group):
    """One head's key and value rows [..., D] with the rule for values that do not fit:
    (key codes, step, lo), (value codes, step, lo)."""
    kq, vq = list(quantise(k, group)), list(quantise(v, group))
    bad = ~((np.abs(k) <= MAX_ABS) & (np.abs(v) <= MAX_ABS)).all(-1)
    for i, fill in enumerate((0, np.nan, np.nan)):
        kq[i] = np.where(bad[..., None], np.array(fill, kq[i].dtype), kq[i])
    for i in range(3):
        vq[i] = np.where(bad[..., None], np.array(0, vq[i].dtype), vq[i])
    return kq, vq


def dequantise(q, step, lo):
    """q*step + lo, rounded once to float32."""
    group = q.shape[-1] // step.shape[-1]
    s = np.repeat(step.astype(np.float64), group, -1)
    return (q.astype(np.float64) * s + np.repeat(lo.astype(np.float64), group, -1)).astype(np.float32)


def block_bytes(page, dim, group):
    return page * dim + 8 * page * (dim // group)


def key_place(dim, t, c):
    """(byte in the block, shift) of channel c of token t."""
    j, kb, i = c // 32, c % 32 // 8, c % 8
    slot = NIBBLE_ORDER.index(i)
    return t * (dim // 2) + 4 * (kb * (dim // 32) + j) + slot // 2, 4 * (slot % 2)


def value_place(page, dim, t, c):
    b, m, half = c // 32, c % 16, c % 32 // 16
    return page * (dim // 2) + ((t // 4) * 16 + m) * (dim // 8) + 4 * b + t % 4, 4 * half


class Cache:
    """A pool of pages as bytes [n_pages, heads, block]."""

    def __init__(self, n_pages, heads, dim, group, page, fill=0):
        self.heads, self.dim, self.group, self.page = heads, dim, group, page
        self.bytes = np.full((n_pages, heads, block_bytes(page, dim, group)), fill, np.uint8)
        c = np.arange(dim)
        self.kp = [np.array([key_place(dim, t, x) for x in c]).T for t in range(page)]
        self.vp = [np.array([value_place(page, dim, t, x) for x in c]).T for t in range(page)]

    def pair_at(self, value, t):
        n = self.dim // self.group
        return self.page * self.dim + (4 * self.page * n if value else 0) + 4 * n * t

    def write(self, pg, slot, k, v):
        """Token rows k, v [heads, D] into a slot."""
        n = 4 * (self.dim // self.group)
        for value, (place, (q, step, lo)) in enumerate(zip((self.kp, self.vp), quantise_token(k, v, self.group))):
            at, shift = place[slot]
            for s in (0, 4):
                on = shift == s
                keep = self.bytes[pg][:, at[on]] & (0xF0 if s == 0 else 0x0F)
                self.bytes[pg][:, at[on]] = keep | (q[:, on] << s).astype(np.uint8)
            pair = np.stack((step, lo), -1).astype(np.float16).reshape(self.heads, -1).view(np.uint8)
            p = self.pair_at(value, slot)
            self.bytes[pg][:, p:p + n] = pair

    def read(self, pg, slot):
        """Token rows (k, v) [heads, D] float32; NaN where the key pairs are."""
        out = []
        for value, place in enumerate((self.kp, self.vp)):
            at, shift = place[slot]
            q = (self.bytes[pg][:, at] >> shift) & 15
            p = self.pair_at(value, slot)
            pair = np.ascontiguousarray(self.bytes[pg][:, p:p + 4 * (self.dim // self.group)]).view(np.float16)
            pair = pair.reshape(self.heads, -1, 2)
            out.append(dequantise(q, pair[..., 0], pair[..., 1]))
        lost = np.isnan(out[0])
        out[1] = np.where(lost, np.float32(np.nan), out[1])
        return out


def sequences(rows, batch, row_start, kv_len, table, page):
    """(first row, rows, length) of each sequence, bounded as the library bounds them."""
    out = []
    for b in range(batch):
        if row_start is None:
            r0, n = b * (rows // batch), rows // batch
        else:
            r0 = min(max(int(row_start[b]), 0), rows)
            n = min(max(int(row_start[b + 1]), r0), rows) - r0
        out.append((r0, n, min(max(int(kv_len[b]), 0), table.shape[1] * page)))
    return out


def append(cache, k, v, row_start, kv_len, table):
    for b, (r0, n, length) in enumerate(sequences(len(k), len(kv_len), row_start, kv_len, table, cache.page)):
        for i in range(n):
            p = length - n + i
            if p < 0:
                continue
            pg = int(table[b, p // cache.page])
            if 0 <= pg < len(cache.bytes):
                cache.write(pg, p % cache.page, k[r0 + i], v[r0 + i])


def read(cache, rows, row_start, kv_len, table, fill=0.0):
    k = np.full((rows, cache.heads, cache.dim), fill, np.float32)
    v = k.copy()
    for b, (r0, n, length) in enumerate(sequences(rows, len(kv_len), row_start, kv_len, table, cache.page)):
        for i in range(n):
            p = length - n + i
            k[r0 + i] = v[r0 + i] = 0.0
            if p < 0:
                continue
            pg = int(table[b, p // cache.page])
            if 0 <= pg < len(cache.bytes):
                k[r0 + i], v[r0 + i] = cache.read(pg, p % cache.page)
    return k, v


def attention(cache, q, row_start, kv_len, table, scale=None, causal=True, window=0, fill=0.0, spread=None):
    """(O, lse, A, E) in float64.  A = sum_t p_t |v'_t| and E, the largest bound on
    a visible score's float32 error (see test_gpu_kv.py), are for tolerances."""
    rows, q_heads, dim = q.shape
    per = q_heads // cache.heads
    scale = dim ** -0.5 if scale is None else scale
    o = np.full(q.shape, fill, np.float64)
    a = np.zeros(q.shape, np.float64)
    lse = np.full(q.shape[:2], fill, np.float64)
    err = np.zeros(q.shape[:2], np.float64)
    for b, (r0, n, length) in enumerate(sequences(rows, len(kv_len), row_start, kv_len, table, cache.page)):
        if n == 0:
            continue
        pg = [int(table[b, t // cache.page]) for t in range(length)]
        real = [t for t in range(length) if 0 <= pg[t] < len(cache.bytes)]
        got = [cache.read(pg[t], t % cache.page) for t in real]
        kk = np.array([g[0] for g in got], np.float64).reshape(len(real), cache.heads, dim)
        vv = np.array([g[1] for g in got], np.float64).reshape(len(real), cache.heads, dim)
        real = np.array(real, int)
        steps = np.zeros((len(real), cache.heads, dim))
        if spread is not None and len(real):
            for x, t in enumerate(real):
                p = cache.pair_at(0, t % cache.page)
                pair = np.ascontiguousarray(cache.bytes[pg[t]][:, p:p + 4 * (dim // cache.group)]).view(np.float16)
                steps[x] = np.repeat(pair.reshape(cache.heads, -1, 2)[..., 0].astype(np.float64), cache.group, -1)
        for i in range(n):
            pos = length - n + i
            see = np.ones(len(real), bool)
            if causal:
                see &= real <= pos
            if window:
                see &= real > pos - window
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
