"""Attention over the 4-bit cache with sinks and with a shared prefix, against the oracle.

Tolerances as derived in test_gpu_kv.py.  A join of a prefix's sums with the others' adds, in
float32, one exp2 (2^-22, of a factor that numerator and denominator share), a product, a
product-and-sum and their roundings: 8 * 2^-24 of A and 2^-22 of the sum (an addend of lse)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv_oracle as kv
from oracle import kv_step_oracle as step
from tests.gpu_util import say
from tests.test_gpu_kv import SIZES, TYPES, filled, ints, pool, queries, table_for, values
from tests.test_gpu_kv_step import angles, check_bytes, check_queries, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (load anew: a test that reloads the module puts back a library that knows the classes of before)
    awq.load()
    return awq


def check(q, dtype, cache, got, lse, start, lengths, table, **kw):
    def spread(steps, key, x):   # bound on the float32 error of q.k' of each token
        mass = np.abs(x).sum() * (2 * 16 + 15)
        g = cache.group
        return (steps * (g * 2.0 ** -24 * mass)).reshape(len(steps), -1, g)[..., 0].sum(-1) + 6 * 2.0 ** -24 * (np.abs(key) @ np.abs(x))

    o, want_lse, a, err = step.attention(cache, q, start, lengths, table, spread=spread, **kw)
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    n = max(1, max(lengths))
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    tol = a * (2.0 ** -10 + 2.0 ** -17 + 2 * err[..., None] + (2 * n + 8) * 2.0 ** -24)
    tol = tol + half * (np.abs(o) + tol) + 1e-30
    assert np.array_equal(np.isnan(got), np.isnan(o))
    bad = ~(np.abs(got - o) <= tol) & ~np.isnan(o)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4], np.broadcast_to(tol, o.shape)[bad][:4])
    assert np.array_equal(np.isnan(lse), np.isnan(want_lse))
    assert np.array_equal(np.isneginf(lse), np.isneginf(want_lse))
    fine = np.isfinite(want_lse)
    off = np.abs(lse[fine] - want_lse[fine])
    assert (off <= err[fine] + 2.0 ** -22 * (np.abs(want_lse[fine]) + 2)).all(), off.max()


def attend(awq, q, dtype, cache, start, lengths, table, fill=0.0, prefix=None, **kw):
    """Output and lse of the library, in buffers that were filled beforehand, its workspace NaN and with a guard behind it."""
    qd = torch.from_numpy(q.astype(np.float32)).to(TYPES[dtype]).cuda()
    dev = pool(awq, cache)
    out = torch.full(q.shape, fill, dtype=TYPES[dtype], device="cuda")
    size = awq.kv_attention_workspace_size(dev, q.shape[1], len(q), len(lengths), table.shape[1], start is not None,
                                           kw.get("max_rows"), prefix_pages=0 if prefix is None else len(prefix[0]))
    room = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    got = awq.kv_attention(qd, dev, ints(table), ints(lengths), row_start=ints(start), out=out, workspace=room[:size], want_lse=True,
                           prefix=None if prefix is None else (ints(prefix[0]), ints([prefix[1]])), **kw)
    torch.cuda.synchronize()
    assert (room[size:] == 0xFF).all()
    return got


def spoil_unseen(c, table, start, lengths, window, sinks, prefix=None):
    """NaN bytes in every slot that no row sees."""
    used = np.zeros((len(c.bytes), c.page), bool)
    common = prefix[1] if prefix is not None else 0
    for b, length in enumerate(lengths):
        n = int(start[b + 1] - start[b]) if start is not None else 1
        for i in range(n):
            t = np.arange(length)
            for x in t[step.sees(length - n + i, t, True, window, sinks)]:
                pg = int(prefix[0][x // c.page] if x < common else table[b, x // c.page])
                if 0 <= pg < len(used):
                    used[pg, x % c.page] = True
    for t in range(common):
        used[prefix[0][t // c.page], t % c.page] = True
    n = 4 * (c.dim // c.group)
    for pg, slot in zip(*np.nonzero(~used)):
        for value in (0, 1):
            at = c.pair_at(value, slot)
            c.bytes[pg][:, at:at + n] = 0xFF


# ---- sinks ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,page", SIZES)
@pytest.mark.parametrize("window,sinks", [(1, 1), (33, 4), (64, 32), (100, 65), (31, 1 << 40), (1000, 5)])
def test_sinks_of_single_tokens(awq, dim, group, page, dtype, window, sinks):
    """Lengths from nothing on: sinks next to the window, apart from it, within it and past it."""
    rng = np.random.default_rng(dim * 3 + group + page + window)
    heads, per = 2, 3
    lengths = [1, 0, 31, 32, 33, 700, 129, 64, 98, 97, 450, 165]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil_unseen(cache, table, None, lengths, window, sinks)
    q = queries(rng, (len(lengths), heads * per, dim), dtype)
    say("sinks", dim, group, page, dtype, window, sinks)
    got, lse = attend(awq, q, dtype, cache, None, lengths, table, window=window, sinks=sinks)
    check(q, dtype, cache, got, lse, None, lengths, table, window=window, sinks=sinks)


@pytest.mark.parametrize("dim,group,dtype", [(64, 32, "bf16"), (64, 64, "fp16"), (128, 32, "fp16"), (128, 64, "bf16"),
                                             (128, 128, "bf16"), (256, 32, "bf16"), (256, 64, "fp16"), (256, 128, "bf16")])
@pytest.mark.parametrize("window,sinks", [(200, 3), (1, 64), (70, 300), (500, 129)])
def test_sinks_of_ragged_rows(awq, dim, group, dtype, window, sinks):
    """Chunks on the wide path with pieces that are joined, drafts, single tokens, sequences with more rows than
    positions and without tokens; rows behind the last sequence stay."""
    rng = np.random.default_rng(dim + group + window)
    heads, per, page = 2, 3, 16
    lengths = [1300, 1, 0, 90, 700, 0, 515, 301]
    counts = [97, 1, 0, 93, 1, 40, 129, 5]
    table, n_pages = table_for(lengths, page, rng, extra=3)
    cache = filled(rng, n_pages, heads, dim, group, page)
    start = np.concatenate(([0], np.cumsum(counts)))
    spoil_unseen(cache, table, start, lengths, window, sinks)
    q = queries(rng, (int(start[-1]) + 3, heads * per, dim), dtype)
    say("sinks of chunks", dim, group, dtype, window, sinks)
    got, lse = attend(awq, q, dtype, cache, start, lengths, table, fill=5.0, window=window, sinks=sinks, max_rows=129)
    last = int(start[-1])
    assert (got[last:] == 5.0).all()
    check(q[:last], dtype, cache, got[:last], lse[:last], start, lengths, table, window=window, sinks=sinks)


@pytest.mark.parametrize("rows,per", [(3, 4), (5, 4), (13, 4), (40, 3)])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
def test_sinks_of_several_rows(awq, rows, per, dim, group):
    """Drafts and small chunks: 1, 2 and 4 column tiles, and the wide path, without a table of rows."""
    rng = np.random.default_rng(rows + per + dim)
    heads, page, window, sinks = 2, 16, 50, 37
    lengths = [rows, 300, max(0, rows - 2), 0, 77, 481]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    start = np.arange(len(lengths) + 1) * rows
    spoil_unseen(cache, table, start, lengths, window, sinks)
    q = queries(rng, (rows * len(lengths), heads * per, dim), "fp16")
    say("sinks of rows", rows, per, dim)
    got, lse = attend(awq, q, "fp16", cache, None, lengths, table, window=window, sinks=sinks)
    check(q, "fp16", cache, got, lse, None, lengths, table, window=window, sinks=sinks)


@pytest.mark.parametrize("rows", [1, 40])
def test_sinks_with_pages_given_up_between(awq, rows):
    """The pages between the sinks and the window are gone, and some of the sinks' own."""
    rng = np.random.default_rng(3)
    heads, per, dim, group, page, window, sinks = 2, 8, 128, 64, 16, 100, 40
    lengths = [700, 330, 64]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    table[0, 3:(700 - rows - window) // page] = -1
    table[1, 1:3] = [n_pages, -7]
    table[2, :3] = -1
    q = queries(rng, (rows * 3, heads * per, dim), "bf16")
    say("sinks without pages", rows)
    got, lse = attend(awq, q, "bf16", cache, None, lengths, table, window=window, sinks=sinks)
    check(q, "bf16", cache, got, lse, None, lengths, table, window=window, sinks=sinks)


def test_long_stream_with_sinks(awq):
    """A position far beyond the window; every other slot of the stream was never written."""
    rng = np.random.default_rng(9)
    heads, per, dim, group, page, length, window, sinks = 2, 4, 128, 128, 64, 131072 - 5, 1024, 4
    cache = filled(rng, 20, heads, dim, group, page)
    table = np.full((1, 2048), -1)
    table[0, 0] = 0
    at = (length - window) // page
    table[0, at:] = 1 + np.arange(2048 - at) % 19
    q = queries(rng, (1, heads * per, dim), "bf16")
    say("long stream")
    got, lse = attend(awq, q, "bf16", cache, None, [length], table, window=window, sinks=sinks)
    check(q, "bf16", cache, got, lse, None, [length], table, window=window, sinks=sinks)


def test_no_sinks_is_the_window_alone(awq):
    rng = np.random.default_rng(10)
    lengths = [300, 40]
    table, n_pages = table_for(lengths, 16, rng)
    dev = pool(awq, filled(rng, n_pages, 2, 64, 32, 16))
    q = torch.from_numpy(queries(rng, (60, 8, 64), "bf16")).bfloat16().cuda()
    say("no sinks")
    a = awq.kv_attention(q, dev, ints(table), ints(lengths), window=70, sinks=0, want_lse=True)
    b = awq.kv_attention(q, dev, ints(table), ints(lengths), window=70, want_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---- shared prefixes --------------------------------------------------------

def with_prefix(rng, lengths, prefix, page, spare=3):
    """A prefix's table, a page table whose columns before its end hold numbers outside the pool, and the pool's pages."""
    table, n = table_for([max(0, k - prefix // page * page) for k in lengths], page, rng, spare)
    first, common = prefix // page, -(-prefix // page)
    order = rng.permutation(n + common)
    wide = np.full((len(lengths), first + table.shape[1]), 1 << 30)
    wide[:, first:] = np.where(table < n, order[np.minimum(table, n - 1)], 1 << 30)
    return order[n:] if common else np.array([0]), wide, n + common


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,group,page", SIZES)
@pytest.mark.parametrize("prefix", [1, 32, 333, 800])
def test_prefix_of_single_tokens(awq, dim, group, page, dtype, prefix):
    """Sequences behind the prefix, at its end, that end within it, and padded slots; 15 columns or more than a wave's 32."""
    rng = np.random.default_rng(dim * 3 + group + page + prefix)
    heads, per = 2, 3 if page == 16 else 9
    lengths = [prefix + 1, 0, prefix, prefix + 40, prefix + 500, max(1, prefix - 20), prefix + 17, prefix + 33]
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    cache = filled(rng, n_pages, heads, dim, group, page)
    spoil_unseen(cache, table, None, lengths, 0, 0, (ptable, prefix))
    q = queries(rng, (len(lengths), heads * per, dim), dtype)
    say("prefix", dim, group, page, dtype, prefix)
    got, lse = attend(awq, q, dtype, cache, None, lengths, table, prefix=(ptable, prefix))
    check(q, dtype, cache, got, lse, None, lengths, table, prefix=(ptable, prefix))


@pytest.mark.parametrize("dim,group,dtype", [(64, 32, "bf16"), (64, 64, "fp16"), (128, 32, "fp16"), (128, 64, "bf16"),
                                             (128, 128, "bf16"), (256, 32, "bf16"), (256, 64, "fp16"), (256, 128, "bf16")])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("prefix", [90, 600])
def test_prefix_of_ragged_rows(awq, dim, group, dtype, causal, prefix):
    """Chunks, drafts, single tokens, rows within the prefix and without a position, sequences without rows or tokens;
    rows behind the last sequence stay."""
    rng = np.random.default_rng(dim + group + prefix)
    heads, per, page = 2, 3, 16
    lengths = [prefix + 700, prefix + 1, 0, 50, prefix + 300, 0, prefix + 60, prefix + 5]
    counts = [97, 1, 0, 53, 1, 40, 129, 5]
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    cache = filled(rng, n_pages, heads, dim, group, page)
    start = np.concatenate(([0], np.cumsum(counts)))
    q = queries(rng, (int(start[-1]) + 3, heads * per, dim), dtype)
    say("prefix of chunks", dim, group, dtype, causal, prefix)
    got, lse = attend(awq, q, dtype, cache, start, lengths, table, fill=5.0, causal=causal, prefix=(ptable, prefix), max_rows=129)
    last = int(start[-1])
    assert (got[last:] == 5.0).all()
    check(q[:last], dtype, cache, got[:last], lse[:last], start, lengths, table, causal=causal, prefix=(ptable, prefix))


@pytest.mark.parametrize("prefix,pages", [(0, 1), (-5, 2), (1 << 30, 3)])
@pytest.mark.parametrize("rows", [1, 30])
def test_prefix_lengths_are_bounded(awq, prefix, pages, rows):
    """None, and more than the prefix's table holds."""
    rng = np.random.default_rng(5)
    heads, per, dim, group, page = 2, 4, 128, 64, 32
    lengths = [200, 96, 97, 0]
    table, n_pages = table_for(lengths, page, rng)
    cache = filled(rng, n_pages, heads, dim, group, page)
    ptable = table[0, :pages]
    q = queries(rng, (4 * rows, heads * per, dim), "bf16")
    say("prefix bounded", prefix, rows)
    got, lse = attend(awq, q, "bf16", cache, None, lengths, table, prefix=(ptable, prefix))
    check(q, "bf16", cache, got, lse, None, lengths, table, prefix=(ptable, prefix))


def test_prefix_pages_that_do_not_exist(awq):
    rng = np.random.default_rng(6)
    heads, per, dim, group, page = 1, 8, 64, 32, 16
    lengths, prefix = [120, 100], 96
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    ptable[[1, 4]] = [-1, n_pages]
    cache = filled(rng, n_pages, heads, dim, group, page)
    for rows in (1, 40):
        q = queries(rng, (2 * rows, per, dim), "bf16")
        say("prefix without pages", rows)
        got, lse = attend(awq, q, "bf16", cache, None, lengths, table, prefix=(ptable, prefix))
        check(q, "bf16", cache, got, lse, None, lengths, table, prefix=(ptable, prefix))
    ptable[:] = -1
    got, lse = attend(awq, q, "bf16", cache, None, lengths, table, prefix=(ptable, prefix))
    check(q, "bf16", cache, got, lse, None, lengths, table, prefix=(ptable, prefix))


def test_prefix_with_tokens_stored_as_nan(awq):
    """NaN in the prefix reaches the rows of its head that see it, and only those; in a sequence, that sequence."""
    rng = np.random.default_rng(12)
    heads, per, dim, group, page, prefix = 2, 2, 128, 128, 16, 64
    lengths = [40, 70, 0, 64]
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    cache = filled(rng, n_pages, heads, dim, group, page)
    bad = np.full((heads, dim), np.nan, np.float32)
    good = rng.standard_normal((heads, dim)).astype(np.float32)
    bad[0] = good[0]
    cache.write(ptable[3], 2, bad, good)          # position 50, head 1
    q = queries(rng, (4, heads * per, dim), "fp16")
    say("prefix with NaN")
    got, lse = attend(awq, q, "fp16", cache, None, lengths, table, prefix=(ptable, prefix))
    check(q, "fp16", cache, got, lse, None, lengths, table, prefix=(ptable, prefix))
    assert torch.isnan(got[:, per:]).all(-1).all(-1).tolist() == [False, True, False, True] and torch.isfinite(got[:, :per]).all()


@pytest.mark.parametrize("batch,prefix", [(64, 3000), (200, 1000)])
def test_prefix_of_a_large_batch(awq, batch, prefix):
    """Many rows of a head against the prefix in one product, in units that are cut and joined, against float64 on the
    GPU's own read-back."""
    torch.manual_seed(batch)
    rng = np.random.default_rng(batch)
    heads, per, dim, group, page = 4, 8, 128, 128, 64
    lengths = [int(x) for x in prefix + rng.integers(1, 300, batch)]
    lengths[5] = 0
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    cache = awq.kv_cache(n_pages, heads, dim, group, page)
    cache.pages.copy_(torch.from_numpy(filled(rng, n_pages, heads, dim, group, page).bytes))
    full = table.copy()
    full[:, :prefix // page] = ptable[:prefix // page]
    q = torch.randn(batch, heads * per, dim, device="cuda").bfloat16()
    say("prefix of a batch", batch)
    got, lse = awq.kv_attention(q, cache, ints(table), ints(lengths), prefix=(ints(ptable), ints([prefix])), want_lse=True)
    tail = prefix % page
    shared = awq.kv_read(cache, ints(ptable[None]), ints([prefix]), prefix, dtype=torch.float32)
    for b in range(0, batch, 7):
        if lengths[b] == 0:
            continue
        own = awq.kv_read(cache, ints(full[b:b + 1]), ints([lengths[b]]), lengths[b], dtype=torch.float32)
        kk, vv = (torch.cat((x, y[prefix:])).double() for x, y in zip(shared, own))
        for h in range(0, heads * per, 5):
            s = kk[:, h // per] @ q[b, h].double() * dim ** -0.5
            p = torch.softmax(s, 0)
            want, a = p @ vv[:, h // per], p @ vv[:, h // per].abs()
            e = 128 * 2.0 ** -24 * 47 * q[b, h].double().abs().sum() * dim ** -0.5 * 0.6 + 6 * 2.0 ** -24 * 60   # steps < 0.6
            tol = a * (2.0 ** -10 + 2.0 ** -17 + 2 * e + (2 * lengths[b] + 8) * 2.0 ** -24)
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
            assert ((got[b, h].double() - want).abs() <= tol).all(), (b, h, tail)
            assert abs(lse[b, h].double() - torch.logsumexp(s, 0)) <= e + 2.0 ** -22 * 13
    assert (got[5] == 0).all() and torch.isneginf(lse[5]).all()
    again = awq.kv_attention(q, cache, ints(table), ints(lengths), prefix=(ints(ptable), ints([prefix])), want_lse=True)
    assert torch.equal(again[0], got) and torch.equal(again[1], lse)      # deterministic


@pytest.mark.parametrize("dim,group,dtype", [(64, 64, "bf16"), (128, 32, "fp16"), (256, 64, "bf16")])
def test_prefix_beside_many_sequences(awq, dim, group, dtype):
    """So many sequences that each unit of theirs has a workgroup of its own, few of which have rows for one: the
    prefix is shared out all the same."""
    rng = np.random.default_rng(dim)
    heads, page, batch, prefix = 8, 16, 70, 1500
    counts = [1, 0, 2, 1, 3] * 14
    counts[7], counts[33] = 90, 71
    lengths = [int(prefix + n + rng.integers(0, 40)) for n in counts]
    lengths[5], lengths[11] = 0, 700
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    cache = filled(rng, n_pages, heads, dim, group, page)
    start = np.concatenate(([0], np.cumsum(counts)))
    q = queries(rng, (int(start[-1]), heads, dim), dtype)
    say("prefix beside many", dim)
    got, lse = attend(awq, q, dtype, cache, start, lengths, table, prefix=(ptable, prefix), max_rows=90)
    rows = np.concatenate([np.arange(start[b], start[b + 1]) for b in (0, 2, 5, 7, 11, 33, 69)])     # (the oracle takes its time)
    some, keep = np.concatenate(([0], np.cumsum([counts[b] for b in (0, 2, 5, 7, 11, 33, 69)]))), [0, 2, 5, 7, 11, 33, 69]
    check(q[rows], dtype, cache, got[rows.tolist()], lse[rows.tolist()], some, [lengths[b] for b in keep], table[keep],
          prefix=(ptable, prefix))


@pytest.mark.parametrize("dim,group,dtype", [(64, 64, "fp16"), (128, 128, "bf16"), (256, 32, "fp16")])
def test_prefix_of_many_columns(awq, dim, group, dtype):
    """So many rows and query heads that the join gives each dim/4 threads, with a last workgroup that is not full."""
    rng = np.random.default_rng(dim + 1)
    heads, per, page, batch, prefix = 5, 13, 32, 67, 150
    lengths = [int(prefix + rng.integers(1, 40)) for _ in range(batch)]
    lengths[3], lengths[9] = 0, 100
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    cache = filled(rng, n_pages, heads, dim, group, page)
    q = queries(rng, (batch, heads * per, dim), dtype)
    say("prefix of many columns", dim)
    got, lse = attend(awq, q, dtype, cache, None, lengths, table, prefix=(ptable, prefix))
    keep = [0, 3, 9, 40, 66]
    check(q[keep], dtype, cache, got[keep], lse[keep], None, [lengths[b] for b in keep], table[keep], prefix=(ptable, prefix))


@pytest.mark.parametrize("prefix,most", [(40, 2), (700, 2), (700, 40)])
def test_prefix_beside_a_sequence_with_more_rows_than_said(awq, prefix, most):
    """Its own rows are unspecified; all others are right, and nothing is written behind the workspace."""
    rng = np.random.default_rng(prefix + most)
    heads, per, dim, group, page = 2, 4, 128, 64, 16
    counts = [1, 90, 2, 1]
    lengths = [prefix + 33, prefix + 120, prefix + 7, prefix + 1]
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    cache = filled(rng, n_pages, heads, dim, group, page)
    start = np.concatenate(([0], np.cumsum(counts)))
    q = queries(rng, (int(start[-1]) + 2, heads * per, dim), "bf16")
    say("more rows than said", prefix, most)
    got, lse = attend(awq, q, "bf16", cache, start, lengths, table, fill=5.0, prefix=(ptable, prefix), max_rows=most)
    assert (got[int(start[-1]):] == 5.0).all()
    rows, keep = [0, 91, 92, 93], [0, 2, 3]
    check(q[rows], "bf16", cache, got[rows], lse[rows], [0, 1, 3, 4], [lengths[b] for b in keep], table[keep], prefix=(ptable, prefix))


def test_prefix_scores_far_apart(awq):
    """Either side outweighs the other by far, both ways."""
    rng = np.random.default_rng(15)
    heads, dim, group, page, prefix = 1, 64, 64, 64, 128
    k = rng.standard_normal((256, 1, dim)).astype(np.float32)
    k[:128, 0, 0], k[128:, 0, 0] = -40, 40
    v = rng.standard_normal((256, 1, dim)).astype(np.float32)
    cache = kv.Cache(4, heads, dim, group, page)
    kv.append(cache, k, v, None, [256], np.array([[2, 0, 1, 3]]))
    q = np.zeros((1, 4, dim))
    q[0, 0, 0], q[0, 1, 0], q[0, 2, :] = 8.0, -8.0, -0.5
    ptable, table = np.array([2, 0]), np.array([[-1, -1, 1, 3]])
    for dtype in ("bf16", "fp16"):
        for rows in (1, 30):
            got, lse = attend(awq, np.repeat(q, rows, 0), dtype, cache, None, [256], table, prefix=(ptable, prefix), scale=1.0, causal=False)
            check(np.repeat(q, rows, 0), dtype, cache, got, lse, None, [256], table, prefix=(ptable, prefix), scale=1.0, causal=False)


@pytest.mark.parametrize("rows", [1, 20])
def test_prefix_and_sinks_on_two_streams_at_once(awq, rows):
    """Calls side by side with workspaces of their own, Q and the output as slices: as one after the other."""
    rng = np.random.default_rng(21)
    heads, per, dim, group, page, prefix = 2, 4, 128, 64, 16, 200
    lengths = [prefix + 90, prefix + 3, 0, prefix + 211]
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    table[:, :prefix // page] = ptable[:prefix // page]
    dev = pool(awq, filled(rng, n_pages, heads, dim, group, page))
    big = torch.randn(4 * rows, heads * per + 4, dim, device="cuda").bfloat16()
    q, t, n, shared = big[:, 2:-2], ints(table), ints(lengths), (ints(ptable), ints([prefix]))

    def calls(out):
        return [awq.kv_attention(q, dev, t, n, prefix=shared, want_lse=True, out=out[0][:, :-2])[1],
                awq.kv_attention(q, dev, t, n, window=64, sinks=8, want_lse=True, out=out[1][:, :-2])[1]]

    outs = [[torch.full((4 * rows, heads * per + 2, dim), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(3)]
    say("two streams", rows)
    lses = [calls(outs[0])]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, side in enumerate(sides):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(3):
                last = calls(outs[1 + i])
            lses.append(last)
    torch.cuda.synchronize()
    for i in (1, 2):
        for x in range(2):
            assert torch.equal(outs[i][x], outs[0][x]) and torch.equal(lses[i][x], lses[0][x])
            assert (outs[i][x][:, -2:] == 3.0).all()


# ---- a step as it is used ---------------------------------------------------

@pytest.mark.parametrize("mode", ["sinks", "prefix"])
def test_decoding_steps_captured_in_a_graph(awq, mode):
    """Tables, rotated append and attention, captured once: replays grow the sequences by themselves, and each
    equals the oracle's step."""
    rng = np.random.default_rng(31)
    heads, per, dim, group, page, batch, most = 2, 4, 128, 64, 16, 6, 12
    prefix = 37 if mode == "prefix" else 0
    view = dict(window=20, sinks=5) if mode == "sinks" else {}
    kv_len = np.array([prefix, prefix + 31, prefix + 60, prefix + 15, prefix, prefix + 100])
    first, common = prefix // page, -(-prefix // page)
    cache = filled(rng, 90, heads, dim, group, page)
    pages = rng.permutation(90)
    ptable, pages = pages[:common], pages[common:]
    table = np.full((batch, most), -1)
    for b, n in enumerate(kv_len):
        k = -(-n // page) - first
        table[b, first:first + k], pages = pages[:k], pages[k:]
        table[b, :first] = ptable[:first]
    cs, qw, kw = angles(200, dim), weight(rng, dim), weight(rng, dim)
    dev, count = pool(awq, cache), np.array([1, 1, 1, 2, 0, 1])
    rows = int(count.sum())
    x = torch.zeros(rows, heads * per + 2 * heads, dim, dtype=torch.bfloat16, device="cuda")   # the fused projection's result
    q, k, v = x[:, :heads * per], x[:, heads * per:-heads], x[:, -heads:]
    t, length, counts, free, taken = ints(table), ints(kv_len), ints(count), ints(pages), ints([0])
    csd, qwd, kwd = (torch.from_numpy(y).cuda() for y in (cs, qw, kw))
    shared = (ints(ptable), ints([prefix])) if prefix else None
    i32 = dict(dtype=torch.int32, device="cuda")
    s = awq.KvStep(torch.empty(batch, **i32), torch.empty(batch + 1, **i32), torch.empty(1, **i32), torch.empty(rows, **i32),
                   torch.empty(rows, dtype=torch.int64, device="cuda"))
    out = torch.empty(rows, heads * per, dim, dtype=torch.bfloat16, device="cuda")
    qo = torch.empty_like(out)
    ws = torch.empty(max(1, awq.kv_attention_workspace_size(dev, heads * per, rows, batch, most, True, 2, prefix_pages=len(ptable))),
                     dtype=torch.uint8, device="cuda")

    def run():
        awq.kv_tables(t, length, counts, free, taken, page=page, rows=rows, out=s)
        awq.kv_append_rotated(dev, q, k, v, t, s.kv_len, csd, row_start=s.row_start, q_weight=qwd, k_weight=kwd, out=qo)
        lse = awq.kv_attention(qo, dev, t, s.kv_len, row_start=s.row_start, max_rows=2, out=out, workspace=ws, want_lse=True,
                               prefix=shared, **view)[1]
        length.copy_(s.kv_len)
        taken.copy_(s.taken)
        return lse

    say("step in a graph", mode)
    kept = [y.clone() for y in (t, length, taken, dev.pages)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    for y, z in zip((t, length, taken, dev.pages), kept):
        y.copy_(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lse = run()
    state = (table, kv_len, None, 0)
    oracle_prefix = (ptable, prefix) if prefix else None
    for i in range(12):
        new = torch.from_numpy(rng.standard_normal(x.shape).astype(np.float32)).bfloat16()
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        torch.ones(1000, device="cuda").sum().item()   # (the program's own work between the replays)
        state = step.tables(page, state[1], count, pages, state[3], state[0], rows)
        new = new.float().numpy()
        table, lengths, start = state[0], state[1], state[2]
        step.append_rotated(cache, new[:, :heads * per], new[:, heads * per:-heads], new[:, -heads:], start, lengths, table, cs, qw, kw)
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(s.slot.cpu().numpy(), state[5])
        check_queries(qo, new[:, :heads * per], qw, cs, step.row_positions(rows, start, lengths, table, page))
        check_bytes(dev, cache)
        check(qo.float().cpu().numpy(), "bf16", cache, out, lse, start, lengths, table, prefix=oracle_prefix, **view)


def test_two_graphs_of_a_prefix(awq):
    """Two captured calls with workspaces of their own, replayed in turn; prefix and lengths change between them."""
    rng = np.random.default_rng(33)
    torch.manual_seed(33)
    heads, per, dim, group, page, batch, most = 2, 4, 64, 32, 16, 9, 40
    dev = pool(awq, filled(rng, batch * most, heads, dim, group, page))
    table = torch.from_numpy(rng.permutation(batch * most).reshape(batch, most)).int().cuda()
    ptable, plen, length = table[3].clone(), ints([100]), ints([300] * batch)
    graphs = []
    for rows in (1, 12):
        q = torch.randn(batch * rows, heads * per, dim, device="cuda", dtype=torch.float16)
        size = awq.kv_attention_workspace_size(dev, heads * per, batch * rows, batch, most, prefix_pages=most)
        ws, out = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
        awq.kv_attention(q, dev, table, length, prefix=(ptable, plen), out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _, lse = awq.kv_attention(q, dev, table, length, prefix=(ptable, plen), out=out, workspace=ws, want_lse=True)
        graphs.append((graph, q, out, lse, ws))
    say("two graphs")
    for i in range(8):
        graph, q, out, lse, _ = graphs[i % 2]
        plen.fill_(int(rng.integers(0, 500)))
        length.copy_(ints(rng.integers(0, 640, batch)))
        q.copy_(torch.randn(q.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        torch.ones(1000, device="cuda").sum().item()
        want = awq.kv_attention(q, dev, table, length, prefix=(ptable, plen), want_lse=True)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i


def test_bindings_refuse(awq):
    c = awq.kv_cache(4, 2, 64, group=64)
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    table, length, one = ints([[0], [1]]), ints([1, 1]), ints([1])
    ok = dict(Q=q, cache=c, block_table=table, kv_len=length)
    awq.kv_attention(**ok, prefix=(one, one))
    for bad, error in ((dict(sinks=1), awq.AwqError), (dict(sinks=-1, window=4), awq.AwqError), (dict(window=4, prefix=(one, one)), awq.AwqError),
                       (dict(window=4, sinks=1, causal=False), awq.AwqError), (dict(prefix=(table, one)), ValueError),
                       (dict(prefix=(one, length)), ValueError), (dict(prefix=(one.long(), one)), TypeError),
                       (dict(prefix=(one, one.cpu())), ValueError), (dict(prefix=(one[:0], one)), awq.AwqError)):
        with pytest.raises(error):
            awq.kv_attention(**{**ok, **bad})
