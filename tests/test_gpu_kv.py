"""The 4-bit key/value cache on the GPU against the oracle.

Tolerances.  The cache's bytes and what is read back are equal, bit for bit.
Attention, per output, with A = sum_t p_t |v'_t| and 2^-11 the half step of fp16:
  - P is rounded to fp16 (2^-11 of each p; below fp16's normal range 2^-25 of the
    reference, which is at most 2^8 below the largest p: 2^-17 in all) and v' to
    fp16 (2^-11):                                     A * (2^-10 + 2^-17)
  - a score's float32 error e changes p by e, the sum of p by e:   A * 2e
  - float32 sums of P*v' and P over n tokens:        A * 2n * 2^-24
  - the output type's rounding:                       half a step of |O|
e: a group's sum adds base + code times q (base 16), `group`
additions of partial sums no larger than (base + 15) * sum |q|; step times it and
lo - base*step times sum q (4 roundings of at most (2*base + 15) * sum |q| * step
beyond |S|) then take the base out.  Both are within group*2^-24*M*step with
M = (2*base + 15) * sum |q| for groups of 32 and more; the groups' float32
combinations add 4 roundings of |S|; scores are in units of log2 (2 more).
lse: e + 2^-22*(|lse| + 1) (exp2, log2 and the sum).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv_oracle as kv
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (load anew: a test that reloads the module puts back a library that knows the classes of before)
    awq.load()
    return awq


def ints(x):
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def table_for(lengths, page, rng, spare=3, extra=0):
    """A page table with shuffled pages; unused entries hold numbers outside the pool."""
    need = [-(-int(n) // page) for n in lengths]
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages)
    t = np.full((len(lengths), max(1, max(need)) + extra), 1 << 30, np.int64)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = order[at:at + k]
        at += k
    return t, n_pages


def values(rng, shape, dtype):
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[-1])) + rng.standard_normal(shape[-1])
    t = torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype])
    return t.float().numpy(), t.cuda()


def pool(awq, cache, shift=0):
    """The oracle's pool on the GPU."""
    return awq.KvCache(torch.from_numpy(cache.bytes.copy()).cuda(), cache.dim, cache.group, cache.page)


def filled(rng, n_pages, heads, dim, group, page):
    """A pool whose every slot holds a token: random codes, steps and lowest values."""
    c = kv.Cache(n_pages, heads, dim, group, page)
    c.bytes[:] = rng.integers(0, 256, c.bytes.shape)
    for value in (0, 1):
        n = page * dim // group
        step = np.exp(rng.standard_normal((n_pages, heads, n)) * 0.3) * 0.15
        lo = -7.5 * step + 0.3 * rng.standard_normal(step.shape)
        at = page * dim + 4 * n * value
        c.bytes[:, :, at:at + 4 * n] = np.stack((step, lo), -1).astype(np.float16).reshape(n_pages, heads, -1).view(np.uint8)
    return c


def spoil(c, table, lengths):
    """NaN bytes (0xFF) in every slot that no sequence's length reaches."""
    used = np.zeros((len(c.bytes), c.page), bool)
    for b, n in enumerate(lengths):
        for t in range(int(n)):
            pg = int(table[b, t // c.page])
            if 0 <= pg < len(used):
                used[pg, t % c.page] = True
    n = 4 * (c.dim // c.group)
    for pg, slot in zip(*np.nonzero(~used)):
        for value in (0, 1):
            at = c.pair_at(value, slot)
            c.bytes[pg][:, at:at + n] = 0xFF


# ---- writing and reading back -----------------------------------------------

SIZES = [(64, 32, 16), (64, 64, 64), (128, 32, 32), (128, 64, 16), (128, 128, 16), (128, 128, 128), (256, 32, 16),
         (256, 64, 256), (256, 128, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dim,group,page", SIZES)
def test_append_then_read_ragged(awq, dim, group, page, dtype):
    """Ragged rows over old tokens: sequences without rows, of one row, longer
    than their positions, on pages that do not exist; rows behind the last sequence."""
    rng = np.random.default_rng(dim + group + page)
    heads = 3
    lengths = [37, 0, 1, 70, 5, 4, 23, 8]
    counts = [33, 0, 1, 1, 9, 4, 2, 6]          # 9 > 5: four rows have no position
    table, n_pages = table_for(lengths, page, rng)
    table[6, :] = n_pages                        # a page behind the pool
    table[3, -(-70 // page) - 1] = -1            # the last token's page is gone
    start = np.concatenate(([0], np.cumsum(counts)))
    rows = int(start[-1]) + 5
    k, kd = values(rng, (rows, heads, dim), dtype)
    v, vd = values(rng, (rows, heads, dim), dtype)
    c = kv.Cache(n_pages, heads, dim, group, page, fill=0xA5)
    dev = pool(awq, c)
    say("append", dim, group, page, dtype)
    awq.kv_append(dev, kd, vd, ints(table), ints(lengths), row_start=ints(start))
    torch.cuda.synchronize()
    kv.append(c, k, v, start, lengths, table)
    assert np.array_equal(dev.pages.cpu().numpy(), c.bytes)      # the rows' slots, and nothing else
    say("read", dim, group, page, dtype)
    out = tuple(torch.full((rows, heads, dim), 7.0, dtype=TYPES[dtype], device="cuda") for _ in range(2))
    awq.kv_read(dev, ints(table), ints(lengths), rows, row_start=ints(start), out=out)
    torch.cuda.synchronize()
    for got, want in zip(out, kv.read(c, rows, start, lengths, table, fill=7.0)):
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(TYPES[dtype]))


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("batch", [63, 64, 65, 700, 4100])
def test_append_and_read_of_many_sequences(awq, batch, dim, group):
    """More sequences than a wave looks at at a time; the first rows belong to none."""
    rng = np.random.default_rng(batch)
    heads, page = 1, 16
    counts = rng.choice([0, 0, 1, 1, 2, 7], batch)
    lengths = [int(n + m) for n, m in zip(counts, rng.choice([0, 1, 5], batch))]
    table, n_pages = table_for(lengths, page, rng)
    start = 3 + np.concatenate(([0], np.cumsum(counts)))
    rows = int(start[-1]) + 2
    k, kd = values(rng, (rows, heads, dim), "fp16")
    v, vd = values(rng, (rows, heads, dim), "fp16")
    c = kv.Cache(n_pages, heads, dim, group, page, fill=0xA5)
    dev = pool(awq, c)
    say("many sequences", batch, dim)
    awq.kv_append(dev, kd, vd, ints(table), ints(lengths), row_start=ints(start))
    torch.cuda.synchronize()
    kv.append(c, k, v, start, lengths, table)
    assert np.array_equal(dev.pages.cpu().numpy(), c.bytes)
    out = tuple(torch.full((rows, heads, dim), 7.0, dtype=torch.float32, device="cuda") for _ in range(2))
    awq.kv_read(dev, ints(table), ints(lengths), rows, row_start=ints(start), out=out)
    for got, want in zip(out, kv.read(c, rows, start, lengths, table, fill=7.0)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("each,lengths", [(1, [1, 2, 3, 4, 5, 64, 0, 17]), (5, [5, 6, 7, 8, 33, 3]), (4, [4, 8, 64]),
                                          (64, [64, 128])])
def test_append_the_same_rows_for_each_sequence(awq, each, lengths):
    rng = np.random.default_rng(each)
    heads, dim, group, page = 5, 128, 64, 16
    table, n_pages = table_for(lengths, page, rng, extra=2)
    rows = each * len(lengths)
    k, kd = values(rng, (rows, heads, dim), "bf16")
    v, vd = values(rng, (rows, heads, dim), "bf16")
    c = kv.Cache(n_pages, heads, dim, group, page)
    dev = awq.kv_cache(n_pages, heads, dim, group, page)
    say("append", each, lengths)
    awq.kv_append(dev, kd, vd, ints(table), ints(lengths))
    got = awq.kv_read(dev, ints(table), ints(lengths), rows, dtype=torch.float32)
    kv.append(c, k, v, None, lengths, table)
    assert np.array_equal(dev.pages.cpu().numpy(), c.bytes)
    for g, want in zip(got, kv.read(c, rows, None, lengths, table)):
        assert np.array_equal(g.cpu().numpy(), want)


def test_append_values_at_the_edges(awq):
    """Constant groups, ties of the rounding, subnormal steps, the largest values, and
    rows that do not fit (a NaN, an infinity, 32769) in the key or the value."""
    rng = np.random.default_rng(3)
    heads, dim, group, page, n = 2, 64, 32, 16, 12
    k = rng.standard_normal((n, heads, dim)).astype(np.float32)
    v = rng.standard_normal((n, heads, dim)).astype(np.float32)
    k[0], v[0] = 2.5, 0.0
    k[1, :, ::2], k[1, :, 1::2] = -32768.0, 32768.0
    v[1] = np.arange(dim) % 31 / 2                                 # step 1: every other one a tie
    k[2], v[2] = 1e-7 * k[2], 3e-5 * v[2]                          # steps at the bottom of fp16
    k[3, 0, 5], v[4, 1, 9], k[5, 1, 63], v[6, 0, 0] = np.nan, np.inf, -np.inf, 32769.0
    k[7], v[7] = -0.0, 1e-30
    k[8], k[8, :, 3], k[8, :, 35] = 0.11847, -181.5, -181.5
    k[8, :, 9], k[8, :, 41] = 5.82421875, 5.82421875                # a step on a tie of fp16
    table, length = np.array([[1]]), [n]
    c = kv.Cache(2, heads, dim, group, page)
    dev = awq.kv_cache(2, heads, dim, group, page)
    awq.kv_append(dev, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), ints(table), ints(length))
    got = awq.kv_read(dev, ints(table), ints(length), n, dtype=torch.float32)
    kv.append(c, k, v, None, length, table)
    assert np.array_equal(dev.pages.cpu().numpy(), c.bytes)
    for g, want in zip(got, kv.read(c, n, None, length, table)):
        assert np.array_equal(g.cpu().numpy(), want, equal_nan=True)
    assert torch.isnan(got[0][3, 0]).all() and torch.isnan(got[1][3, 0]).all()
    assert torch.isfinite(got[0][3, 1]).all()


def test_append_and_read_strided_rows_and_pages(awq):
    """K and V as slices of a fused projection, pages as slices of a larger pool,
    outputs as slices: nothing outside them is written."""
    rng = np.random.default_rng(4)
    heads, dim, group, page, rows = 2, 64, 64, 16, 21
    lengths, table = [40], np.array([[2, 0, 1]])
    k, kd = values(rng, (rows, heads, dim), "fp16")
    v, vd = values(rng, (rows, heads, dim), "fp16")
    fused = torch.zeros(rows, 4 + 2 * heads, dim, dtype=torch.float16, device="cuda")
    fused[:, 4:4 + heads], fused[:, 4 + heads:] = kd, vd
    c = kv.Cache(3, heads, dim, group, page, fill=0x11)
    big = torch.full((3, 5, heads, c.bytes.shape[2]), 0x11, dtype=torch.uint8, device="cuda")
    dev = awq.KvCache(big[:, 3], dim, group, page)
    awq.kv_append(dev, fused[:, 4:4 + heads], fused[:, 4 + heads:], ints(table), ints(lengths))
    out = torch.full((rows, 2 * heads + 1, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    awq.kv_read(dev, ints(table), ints(lengths), rows, out=(out[:, :heads], out[:, heads:2 * heads]))
    kv.append(c, k, v, None, lengths, table)
    assert np.array_equal(big[:, 3].cpu().numpy(), c.bytes)
    assert (big[:, :3] == 0x11).all() and (big[:, 4] == 0x11).all()
    want = kv.read(c, rows, None, lengths, table)
    assert torch.equal(out[:, :heads].cpu(), torch.from_numpy(want[0]).bfloat16())
    assert torch.equal(out[:, heads:2 * heads].cpu(), torch.from_numpy(want[1]).bfloat16())
    assert (out[:, 2 * heads] == 9.0).all()


def test_append_of_four_tokens_and_of_single_ones_agree(awq):
    """Whole 4-token blocks are stored by words, others by bytes: token by token
    and all at once give the same bytes."""
    rng = np.random.default_rng(5)
    heads, dim, group, page, n = 4, 128, 32, 16, 64
    k, kd = values(rng, (n, heads, dim), "bf16")
    v, vd = values(rng, (n, heads, dim), "bf16")
    table = ints([[3, 1, 0, 2]])
    a, b = awq.kv_cache(4, heads, dim, group, page), awq.kv_cache(4, heads, dim, group, page)
    awq.kv_append(a, kd, vd, table, ints([n]))
    for t in range(n):
        awq.kv_append(b, kd[t:t + 1], vd[t:t + 1], table, ints([t + 1]))
    assert torch.equal(a.pages, b.pages)


# ---- attention --------------------------------------------------------------

def check(q, dtype, cache, got, lse, start, lengths, table, fill=0.0, **kw):
    base = 16

    def spread(step, key, x):   # bound on the float32 error of q.k' of each token
        mass = np.abs(x).sum() * (2 * base + 15)
        g = cache.group
        return (step * (g * 2.0 ** -24 * mass)).reshape(len(step), -1, g)[..., 0].sum(-1) \
            + 6 * 2.0 ** -24 * (np.abs(key) @ np.abs(x))

    o, want_lse, a, err = kv.attention(cache, q, start, lengths, table, fill=fill, spread=spread, **kw)
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    n = max(1, max(lengths))
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    tol = a * (2.0 ** -10 + 2.0 ** -17 + 2 * err[..., None] + 2 * n * 2.0 ** -24)
    tol = tol + half * (np.abs(o) + tol) + 1e-30
    assert np.array_equal(np.isnan(got), np.isnan(o))
    bad = ~(np.abs(got - o) <= tol) & ~np.isnan(o)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4], np.broadcast_to(tol, o.shape)[bad][:4])
    assert np.array_equal(np.isnan(lse), np.isnan(want_lse))
    assert np.array_equal(np.isneginf(lse), np.isneginf(want_lse))
    fine = np.isfinite(want_lse)
    off = np.abs(lse[fine] - want_lse[fine])
    assert (off <= err[fine] + 2.0 ** -22 * (np.abs(want_lse[fine]) + 1)).all(), off.max()


def attend(awq, q, dtype, cache, start, lengths, table, fill=0.0, **kw):
    """Output and lse of the library, in buffers that were filled beforehand, its workspace NaN."""
    qd = torch.from_numpy(q.astype(np.float32)).to(TYPES[dtype]).cuda()
    dev = pool(awq, cache)
    out = torch.full(q.shape, fill, dtype=TYPES[dtype], device="cuda")
    size = awq.kv_attention_workspace_size(dev, q.shape[1], len(q), len(lengths), table.shape[1], start is not None,
                                           kw.get("max_rows"))
    ws = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    return awq.kv_attention(qd, dev, ints(table), ints(lengths), row_start=ints(start), out=out, workspace=ws,
                            want_lse=True, **kw)


def queries(rng, shape, dtype):
    return values(rng, shape, dtype)[0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,page", SIZES)
def test_attention_one_token(awq, dim, group, page, dtype):
    """Decoding: lengths from nothing to several workers' shares, shuffled pages,
    NaN in every slot that does not count."""
    rng = np.random.default_rng(dim * 3 + group + page)
    heads, per = 2, 3
    lengths = [1, 0, 31, 32, 33, 700, 129, 16, 17, 450]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil(cache, table, lengths)
    q = queries(rng, (len(lengths), heads * per, dim), dtype)
    say("attend", dim, group, page, dtype)
    got, lse = attend(awq, q, dtype, cache, None, lengths, table)
    check(q, dtype, cache, got, lse, None, lengths, table)


@pytest.mark.parametrize("per", [1, 2, 5, 8, 16, 17, 32, 40, 64, 71])
def test_attention_query_heads_of_a_key_head(awq, per):
    rng = np.random.default_rng(per)
    heads, dim, group, page, lengths = 1, 64, 64, 16, [100, 3, 650]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil(cache, table, lengths)
    q = queries(rng, (3, heads * per, dim), "bf16")
    say("per", per)
    got, lse = attend(awq, q, "bf16", cache, None, lengths, table)
    check(q, "bf16", cache, got, lse, None, lengths, table)


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("rows,per", [(3, 4), (5, 4), (13, 4), (40, 3)])
def test_attention_several_rows(awq, rows, per, dim, group):
    """Draft tokens and small chunks (1, 2 and 4 column tiles, and the wide path):
    causal, sequences shorter than their rows, an empty one."""
    rng = np.random.default_rng(rows + per + dim)
    heads, page = 2, 16
    lengths = [rows, 300, rows - 2, 0, 77, 481]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil(cache, table, lengths)
    q = queries(rng, (rows * len(lengths), heads * per, dim), "fp16")
    say("rows", rows, per, dim)
    got, lse = attend(awq, q, "fp16", cache, None, lengths, table)
    check(q, "fp16", cache, got, lse, None, lengths, table)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 33), (True, 100000)])
@pytest.mark.parametrize("max_rows", [None, 131])
def test_attention_ragged_rows(awq, causal, window, max_rows):
    """Single tokens, drafts and chunks in one call, rows behind the last sequence."""
    rng = np.random.default_rng(7 + window)
    heads, per, dim, group, page = 2, 4, 128, 64, 32
    lengths = [131, 260, 0, 9, 600, 1, 90]
    counts = [131, 1, 0, 9, 20, 1, 95]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil(cache, table, lengths)
    start = np.concatenate(([0], np.cumsum(counts)))
    rows = int(start[-1]) + 7
    q = queries(rng, (rows, heads * per, dim), "bf16")
    say("ragged", causal, window, max_rows)
    got, lse = attend(awq, q, "bf16", cache, start, lengths, table, fill=5.0, causal=causal, window=window,
                      max_rows=max_rows)
    assert (got[int(start[-1]):] == 5.0).all()
    last = int(start[-1])
    check(q[:last], "bf16", cache, got[:last], lse[:last], start, lengths, table, causal=causal, window=window)


@pytest.mark.parametrize("rows", [1, 60])
def test_attention_pages_that_do_not_exist(awq, rows):
    """Page numbers outside the pool, in the middle and everywhere: their positions are left out."""
    rng = np.random.default_rng(11)
    heads, per, dim, group, page = 1, 8, 64, 32, 16
    lengths = [200, 150, 64]
    table, n_pages = table_for(lengths, page, rng)
    table[0, [1, 4, 5]] = [-1, n_pages, 1 << 30]
    table[1, :] = -5
    table[2, 0] = -1
    cache = filled(rng, n_pages, heads, dim, group, page)
    q = queries(rng, (rows * 3, per, dim), "bf16")
    say("missing pages", rows)
    got, lse = attend(awq, q, "bf16", cache, None, lengths, table)
    check(q, "bf16", cache, got, lse, None, lengths, table)
    assert (got[rows:2 * rows] == 0).all() and torch.isneginf(lse[rows:2 * rows]).all()


@pytest.mark.parametrize("rows", [4, 70])
def test_attention_tokens_stored_as_nan(awq, rows):
    """A row that sees a NaN token is NaN; one that does not, by causality, by the window or by
    its head, is untouched."""
    rng = np.random.default_rng(12)
    heads, per, dim, group, page, length = 2, 2, 128, 128, 16, 90
    table = np.array([[0, 1, 2, 3, 4, 5]])
    k = rng.standard_normal((length, heads, dim)).astype(np.float32)
    v = rng.standard_normal((length, heads, dim)).astype(np.float32)
    v[length - 2, 1, 3] = np.inf
    k[length - 40, 0, 9] = np.nan
    cache = kv.Cache(6, heads, dim, group, page)
    kv.append(cache, k, v, None, [length], table)
    q = queries(rng, (rows, heads * per, dim), "fp16")
    for window in (0, 30):
        got, lse = attend(awq, q, "fp16", cache, None, [length], table, window=window)
        check(q, "fp16", cache, got, lse, None, [length], table, window=window)
        assert torch.isnan(got[-1, per:]).all() and torch.isfinite(got[-3, per:]).all()
        assert torch.isfinite(got[-1, :per]).all() == (window == 30)


def test_attention_of_extreme_scores(awq):
    """Scores that rise along the sequence by far more than the softmax's lag, that are
    all very low, and a query of zeros."""
    rng = np.random.default_rng(13)
    heads, dim, group, page, length = 1, 64, 64, 64, 900
    table = np.arange(15)[None]
    k = rng.standard_normal((length, 1, dim)).astype(np.float32)
    k[:, 0, 0] = np.linspace(-60, 60, length)
    v = rng.standard_normal((length, 1, dim)).astype(np.float32)
    cache = kv.Cache(15, heads, dim, group, page)
    kv.append(cache, k, v, None, [length], table)
    q = np.zeros((1, 4, dim))
    q[0, 0, 0], q[0, 1, 0], q[0, 2, :] = 8.0, -8.0, -0.5
    for dtype in ("bf16", "fp16"):
        got, lse = attend(awq, q, dtype, cache, None, [length], table, scale=1.0)
        check(q, dtype, cache, got, lse, None, [length], table, scale=1.0)


def test_attention_long_sequence(awq):
    """One long sequence shared by every worker, against float64 on the GPU's own read-back."""
    torch.manual_seed(1)
    heads, per, dim, group, page, length = 2, 4, 128, 128, 64, 40003
    n = -(-length // page)
    table = torch.randperm(n, device="cuda").int()[None]
    c = awq.kv_cache(n, heads, dim, group, page)
    k, v = (torch.randn(length, heads, dim, device="cuda") for _ in range(2))
    awq.kv_append(c, k, v, table, ints([length]))
    q = torch.randn(1, heads * per, dim, device="cuda").bfloat16()
    got, lse = awq.kv_attention(q, c, table, ints([length]), want_lse=True)
    kk, vv = (x.double() for x in awq.kv_read(c, table, ints([length]), length, dtype=torch.float32))
    for h in range(heads * per):
        s = kk[:, h // per] @ q[0, h].double() * dim ** -0.5
        p = torch.softmax(s, 0)
        want, a = p @ vv[:, h // per], p @ vv[:, h // per].abs()
        e = 128 * 2.0 ** -24 * 47 * q[0, h].double().abs().sum() * dim ** -0.5 * 0.6 + 6 * 2.0 ** -24 * 60   # steps < 0.6
        tol = a * (2.0 ** -10 + 2.0 ** -17 + 2 * e + 2 * length * 2.0 ** -24)
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
        assert ((got[0, h].double() - want).abs() <= tol).all()
        assert abs(lse[0, h].double() - torch.logsumexp(s, 0)) <= e + 2.0 ** -22 * 12


def test_attention_strides_streams_and_determinism(awq):
    """Q and the output as slices, on a stream of its own, twice: equal bits, and nothing outside written."""
    rng = np.random.default_rng(17)
    heads, per, dim, group, page = 2, 4, 128, 64, 16
    lengths = [900, 5, 333]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    q = queries(rng, (6, heads * per, dim), "bf16")
    dev = pool(awq, cache)
    wide = torch.zeros(6, heads * per + 4, dim, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:-2] = torch.from_numpy(q.astype(np.float32)).bfloat16().cuda()
    outs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t, n = ints(table), ints(lengths)
        for _ in range(2):
            out = torch.full((6, heads * per + 2, dim), 3.0, dtype=torch.bfloat16, device="cuda")
            _, lse = awq.kv_attention(wide[:, 2:-2], dev, t, n, out=out[:, :-2], want_lse=True)
            outs.append((out, lse))
    side.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert (outs[0][0][:, -2:] == 3.0).all()
    check(q, "bf16", cache, outs[0][0][:, :-2], outs[0][1], None, lengths, table)


def test_decoding_step_captured_in_a_graph(awq):
    """Append, then attend, captured once: replays follow the lengths, tables and inputs that
    the program changes between them, and equal the eager calls."""
    rng = np.random.default_rng(19)
    torch.manual_seed(19)
    heads, per, dim, group, page, batch, most = 2, 4, 128, 128, 16, 5, 64
    c, eager = (awq.kv_cache(batch * most, heads, dim, group, page) for _ in range(2))
    table = torch.randperm(batch * most, device="cuda").int().view(batch, most)
    length = ints([0, 200, 15, 700, 31])
    old = 800
    for x in (c, eager):
        torch.manual_seed(3)
        kv0, vv0 = (torch.randn(old, heads, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        awq.kv_append(x, kv0.repeat(batch, 1, 1), vv0.repeat(batch, 1, 1), table, ints([old] * batch))
    q = torch.zeros(batch, heads * per, dim, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros(batch, heads, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    out = torch.zeros_like(q)
    ws = torch.empty(awq.kv_attention_workspace_size(c, heads * per, batch, batch, most), dtype=torch.uint8, device="cuda")

    def step(x, o, w):
        awq.kv_append(x, k, v, table, length)
        return awq.kv_attention(q, x, table, length, out=o, workspace=w, want_lse=True)

    step(c, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse = step(c, out, ws)
    awq.kv_append(eager, k, v, table, length)   # the warm-up's write
    for i in range(4):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        length.add_(ints(rng.integers(0, 40, batch)) + 1)
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = step(eager, torch.empty_like(out), None)
        torch.cuda.synchronize()
        assert torch.equal(c.pages, eager.pages)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dim,group,dtype", [(64, 32, "bf16"), (64, 64, "fp16"), (128, 32, "fp16"), (128, 64, "bf16"),
                                             (128, 128, "bf16"), (256, 32, "bf16"), (256, 64, "fp16"), (256, 128, "bf16")])
@pytest.mark.parametrize("window", [0, 200])
def test_attention_of_few_long_chunks(awq, dim, group, dtype, window):
    """Chunks whose columns and tokens are shared out among workgroups: pieces joined, next to
    sequences without rows, of one row, with more rows than positions, and without tokens."""
    rng = np.random.default_rng(dim + group + window)
    heads, per, page = 2, 3, 16
    lengths = [1300, 1, 0, 90, 700, 0, 515]
    counts = [97, 1, 0, 93, 1, 40, 129]
    table, n_pages = table_for(lengths, page, rng, extra=3)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil(cache, table, lengths)
    start = np.concatenate(([0], np.cumsum(counts)))
    q = queries(rng, (int(start[-1]) + 3, heads * per, dim), dtype)
    say("long chunks", dim, group, dtype, window)
    got, lse = attend(awq, q, dtype, cache, start, lengths, table, fill=5.0, window=window, max_rows=129)
    last = int(start[-1])
    assert (got[last:] == 5.0).all()
    check(q[:last], dtype, cache, got[:last], lse[:last], start, lengths, table, window=window)


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
def test_attention_of_many_chunks(awq, dim, group):
    """So many chunks that each (chunk, head) has a workgroup of its own."""
    rng = np.random.default_rng(dim)
    heads, per, page, batch, rows = 4, 5, 16, 131, 14
    lengths = [int(x) for x in rng.integers(0, 60, batch)]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil(cache, table, lengths)
    q = queries(rng, (batch * rows, heads * per, dim), "bf16")
    say("many chunks", dim)
    got, lse = attend(awq, q, "bf16", cache, None, lengths, table)
    check(q, "bf16", cache, got, lse, None, lengths, table)


@pytest.mark.parametrize("most", [96, 97, 192, 193, 224])
@pytest.mark.parametrize("dim,rows,batch", [(64, 1, 7), (128, 3, 1), (256, 2, 90)])
def test_attention_of_short_sequences(awq, most, dim, rows, batch):
    """Around the lengths up to which no sequence is cut."""
    rng = np.random.default_rng(most + dim)
    heads, per, group, page = 5, 4, 64, 32
    lengths = [int(x) for x in rng.integers(0, most + 1, batch)]
    lengths[0] = most
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil(cache, table, lengths)
    q = queries(rng, (batch * rows, heads * per, dim), "bf16")
    say("short sequences", most, dim, batch)
    got, lse = attend(awq, q, "bf16", cache, None, lengths, table)
    check(q, "bf16", cache, got, lse, None, lengths, table)


@pytest.mark.parametrize("batch", [60, 120])
def test_attention_of_even_chunks(awq, batch):
    """As many chunks of like lengths as a CU takes whole, one or two each; some have no tokens."""
    rng = np.random.default_rng(batch)
    heads, per, dim, group, page, rows = 4, 4, 128, 64, 32, 17
    lengths = [int(x) for x in rng.integers(90, 129, batch)]
    lengths[3] = lengths[batch // 2] = 0
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil(cache, table, lengths)
    q = queries(rng, (batch * rows, heads * per, dim), "fp16")
    say("even chunks", batch)
    got, lse = attend(awq, q, "fp16", cache, None, lengths, table)
    check(q, "fp16", cache, got, lse, None, lengths, table)


@pytest.mark.parametrize("batch", [64, 65, 300])
def test_attention_of_many_sequences(awq, batch):
    """More sequences than one wave looks at at a time, most of them short."""
    rng = np.random.default_rng(batch)
    heads, per, dim, group, page = 3, 4, 128, 64, 16
    lengths = [int(x) for x in np.exp(rng.uniform(-1, 6, batch))]
    lengths[-1] = 900
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil(cache, table, lengths)
    q = queries(rng, (batch, heads * per, dim), "fp16")
    say("many sequences", batch)
    got, lse = attend(awq, q, "fp16", cache, None, lengths, table)
    check(q, "fp16", cache, got, lse, None, lengths, table)


@pytest.mark.parametrize("dim,group,rows", [(64, 64, 1), (128, 128, 6), (256, 32, 1), (64, 32, 90), (128, 32, 90), (256, 128, 90)])
def test_queries_that_are_not_finite_keep_to_themselves(awq, dim, group, rows):
    """A NaN in one query, infinities in another: those are not finite, every other one is as it was."""
    rng = np.random.default_rng(dim + rows)
    heads, per, page, batch = 2, 4, 16, 3
    lengths = [700, 95, 240]
    table, n_pages = table_for(lengths, page, rng)
    dev = pool(awq, filled(rng, n_pages, heads, dim, group, page))
    q = torch.from_numpy(queries(rng, (batch * rows, heads * per, dim), "bf16")).bfloat16().cuda()
    bad = q.clone()
    nan, inf = (0, 3), (batch * rows - 1, 6)
    bad[nan][5] = float("nan")
    bad[inf][7], bad[inf][40] = float("inf"), -float("inf")
    say("queries", dim, rows)
    (o, lse), (po, plse) = (awq.kv_attention(x, dev, ints(table), ints(lengths), want_lse=True) for x in (q, bad))
    assert torch.isfinite(o).all()
    assert torch.isnan(po[nan]).all() and torch.isnan(plse[nan]) and not torch.isfinite(plse[inf])
    for at in (nan, inf):
        po[at], plse[at] = o[at], lse[at]
    assert torch.equal(po, o) and torch.equal(plse, lse)


def test_pages_far_apart(awq):
    """Pages so far apart that offsets into the pool pass 2^32, written, read and attended to."""
    rng = np.random.default_rng(23)
    heads, per, dim, group, page, n = 2, 4, 128, 64, 16, 7
    block = page * dim + 8 * page * (dim // group)
    apart = (5 << 30) // (n - 1) // 16 * 16
    far = torch.empty(apart * (n - 1) + heads * block, dtype=torch.uint8, device="cuda")
    pages = far.as_strided((n, heads, block), (apart, block, 1))
    pages.zero_()
    dev, near = awq.KvCache(pages, dim, group, page), awq.kv_cache(n, heads, dim, group, page)
    table, lengths = np.array([[6, 0, 5], [4, 1, 3]]), [45, 48]
    rows = 45
    k, v = (torch.randn(2 * rows, heads, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(2 * rows, heads * per, dim, device="cuda", dtype=torch.bfloat16)
    results = []
    for x in (dev, near):
        awq.kv_append(x, k, v, ints(table), ints(lengths))
        one = torch.randn(2, heads * per, dim, device="cuda", dtype=torch.bfloat16, generator=torch.Generator("cuda").manual_seed(1))
        results.append((x.pages.contiguous(), *awq.kv_read(x, ints(table), ints(lengths), 2 * rows),
                        *awq.kv_attention(q, x, ints(table), ints(lengths), want_lse=True),
                        *awq.kv_attention(one, x, ints(table), ints(lengths), want_lse=True)))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert (results[0][0] != 0).any(-1).any(-1).tolist() == [True, True, False, True, True, True, True]


def test_chunk_captured_in_a_graph(awq):
    """A ragged chunk and its attention, with joined pieces, captured twice with workspaces of their
    own: replays in turn follow the tables that the program changes, and equal the eager calls."""
    torch.manual_seed(29)
    rng = np.random.default_rng(29)
    heads, per, dim, group, page, batch, most, rows = 2, 4, 128, 64, 16, 3, 90, 250
    c, eager = (awq.kv_cache(batch * most, heads, dim, group, page) for _ in range(2))
    table = torch.randperm(batch * most, device="cuda").int().view(batch, most)
    length, start = ints([300, 60, 9]), ints([0, 200, 201, 210])
    old = torch.randn(2, 1200, heads, dim, device="cuda", dtype=torch.bfloat16)
    for x in (c, eager):
        awq.kv_append(x, old[0].repeat(batch, 1, 1), old[1].repeat(batch, 1, 1), table, ints([1200] * batch))
    q = torch.zeros(rows, heads * per, dim, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros(rows, heads, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    size = awq.kv_attention_workspace_size(c, heads * per, rows, batch, most, True, 240)
    assert size > 0

    def step(x, o, w):
        awq.kv_append(x, k, v, table, length, row_start=start)
        return awq.kv_attention(q, x, table, length, row_start=start, max_rows=240, out=o, workspace=w, want_lse=True)

    graphs = []
    for _ in range(2):
        out, ws = torch.zeros_like(q), torch.empty(size, dtype=torch.uint8, device="cuda")
        step(c, out, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _, lse = step(c, out, ws)
        graphs.append((graph, out, lse, ws))   # (a graph's workspace has to live as long as the graph)
    awq.kv_append(eager, k, v, table, length, row_start=start)   # the warm-ups' write
    for i in range(6):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        counts = rng.integers(0, 80, 3)
        counts[i % 3] = 1 + 80 * (i % 4) // 3
        start.copy_(ints(np.concatenate(([0], np.cumsum(counts)))))
        length.copy_(ints(np.maximum(counts, rng.integers(0, 1200, 3))))
        graph, out, lse, _ = graphs[i % 2]
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = step(eager, torch.empty_like(out), None)
        torch.cuda.synchronize()
        n = int(counts.sum())
        assert torch.equal(c.pages, eager.pages)
        assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], want_lse[:n])


def test_generation_through_the_cache(awq):
    """A prompt, then single tokens, then drafts: each step's rows equal one pass over all rows."""
    rng = np.random.default_rng(23)
    heads, per, dim, group, page, total = 2, 8, 64, 32, 16, 150
    k, kd = values(rng, (total, heads, dim), "bf16")
    v, vd = values(rng, (total, heads, dim), "bf16")
    q = queries(rng, (total, heads * per, dim), "bf16")
    qd = torch.from_numpy(q.astype(np.float32)).bfloat16().cuda()
    table = np.array([[7, 3, 9, 0, 1, 2, 8, 5, 4, 6]])
    c = awq.kv_cache(10, heads, dim, group, page)
    at, outs, lses = 0, [], []
    for n in (100, 1, 1, 1, 5, 3, 1, 38):
        awq.kv_append(c, kd[at:at + n], vd[at:at + n], ints(table), ints([at + n]))
        o, lse = awq.kv_attention(qd[at:at + n], c, ints(table), ints([at + n]), want_lse=True)
        outs.append(o), lses.append(lse)
        at += n
    assert at == total
    cache = kv.Cache(10, heads, dim, group, page)
    kv.append(cache, k, v, None, [total], table)
    assert np.array_equal(c.pages.cpu().numpy()[table[0]], cache.bytes[table[0]])
    check(q, "bf16", cache, torch.cat(outs), torch.cat(lses), None, [total], table)


def test_no_rows(awq):
    c = awq.kv_cache(1, 2, 64, 64, 16)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    table, n = ints([[0], [0]]), ints([3, 0])
    awq.kv_append(c, e, e, table, n)
    k, v = awq.kv_read(c, table, n, 0)
    assert k.shape == v.shape == (0, 2, 64)
    assert awq.kv_attention(e, c, table, n).shape == (0, 2, 64)


def test_python_refuses_mismatches(awq):
    c = awq.kv_cache(2, 2, 64, 64, 16)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    t, n = ints([[0], [1]]), ints([1, 1])
    for call in (lambda: awq.kv_append(c, x, x[:, :1], t, n), lambda: awq.kv_append(c, x, x.float(), t, n),
                 lambda: awq.kv_append(c, x, x, t.long(), n), lambda: awq.kv_append(c, x, x, t, n[:1]),
                 lambda: awq.kv_append(c, x, x, t.cpu(), n), lambda: awq.kv_append(c, x.cpu(), x.cpu(), t, n),
                 lambda: awq.kv_append(c, x, x, t, n, row_start=n), lambda: awq.kv_attention(x.float(), c, t, n),
                 lambda: awq.kv_attention(x, c, t, n, out=x.half()), lambda: awq.kv_append(c, x.int(), x.int(), t, n),
                 lambda: awq.kv_attention(x, c, t, n, workspace=torch.zeros(8, device="cuda")),
                 lambda: awq.kv_append(c, x.transpose(0, 1), x.transpose(0, 1), t, n),
                 lambda: awq.kv_read(c, t, n, 3), lambda: awq.kv_attention(x[:1], c, t, n)):
        with pytest.raises((TypeError, ValueError, awq.AwqError)):
            call()
