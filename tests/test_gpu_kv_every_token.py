"""Each position counts once: attention whose scores are all equal, over values that say which position they are.

Queries are zero, so every score is exactly 0, the reference is -7, every weight 2^7 and every sum of weights an integer
times 2^7, exact. Position t holds 15 in channel t mod p (a prime below the head's dim) and 0 elsewhere, which the cache
holds exactly (lo 0, step 1). So channel c of the output is 15 * (positions seen with t mod p = c) / (positions seen),
rounded by the reciprocal and a product (3 * 2^-24) and to the type (2^-8): times n / 15 that is within 0.5 of the whole
number while that is below 120, and lse is ln n within 2^-22 (|lse| + 2). A position that is dropped or doubled moves one channel
by 1; a tile moves 32 and more. NaN in the prefix is tested on the wide path, too."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_kv import TYPES, filled, ints, queries
from tests.test_gpu_kv_view import attend, check, with_prefix

pytestmark = pytest.mark.gpu

PRIME = {64: 61, 128: 127, 256: 251}


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (load anew: a test that reloads the module puts back a library that knows the classes of before)
    awq.load()
    return awq


def hot(positions, heads, dim):
    x = torch.zeros(len(positions), heads, dim, device="cuda")
    x[torch.arange(len(positions)), :, torch.from_numpy(positions % PRIME[dim]).cuda()] = 15.0
    return x


def count_check(awq, dtype, dim, group, heads, per, page, lengths, counts, prefix=0, causal=True, window=0, sinks=0, most=None):
    rng = np.random.default_rng(sum(lengths) + dim)
    torch.manual_seed(dim)
    batch, p = len(lengths), PRIME[dim]
    first = prefix // page
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    cache = awq.kv_cache(n_pages, heads, dim, group, page)
    own = [np.arange(min(first * page, n), n) for n in lengths]
    at = np.concatenate(own)
    awq.kv_append(cache, torch.randn(len(at), heads, dim, device="cuda"), hot(at, heads, dim), ints(table), ints(lengths),
                  row_start=ints(np.concatenate(([0], np.cumsum([len(x) for x in own])))))
    if prefix:
        awq.kv_append(cache, torch.randn(prefix, heads, dim, device="cuda"), hot(np.arange(prefix), heads, dim), ints(ptable[None]),
                      ints([prefix]))
    start, rows = np.concatenate(([0], np.cumsum(counts))), sum(counts)
    q = torch.zeros(rows, heads * per, dim, dtype=TYPES[dtype], device="cuda")
    even = min(counts) == max(counts) and most is None
    say("every token", dtype, dim, group, batch, rows, prefix, causal, window, sinks)
    got, lse = awq.kv_attention(q, cache, ints(table), ints(lengths), row_start=None if even else ints(start),
                                max_rows=None if even else most or max(counts), causal=causal, window=window, sinks=sinks, want_lse=True,
                                prefix=(ints(ptable), ints([prefix])) if prefix else None)
    b = np.repeat(np.arange(batch), counts)
    length = np.array(lengths)[b]
    pos = length - np.array(counts)[b] + np.arange(rows) - start[b]
    end = pos + 1 if causal else length                       # positions before `end`, ..
    low = np.maximum(pos - window + 1, 0) if window else 0 * pos   # .. from `low` on, and the sinks below it
    end = np.where(pos < 0, 0, end) if causal else end
    sink_end = np.minimum(np.minimum(sinks, low), np.maximum(end, 0)) if window else 0 * pos
    c = np.arange(p)
    upto = lambda x: (x[:, None] - c + p - 1) // p  # noqa: E731  (positions t < x with t mod p = c)
    seen = np.where(end[:, None] > low[:, None], upto(end) - upto(low), 0) + upto(sink_end)
    n = seen.sum(-1)
    assert seen.max() < 120
    seen, n = torch.from_numpy(seen).double().cuda(), torch.from_numpy(n).double().cuda()
    whole = got[..., :p].double() * n[:, None, None] / 15
    bad = torch.nonzero(~((whole - seen[:, None]).abs() < 0.5)).tolist()
    assert len(bad) == 0, (len(bad), bad[:6], [(float(whole[tuple(i)]), float(seen[i[0], i[2]])) for i in bad[:6]])
    assert (got[..., p:] == 0).all()
    some = n > 0
    assert torch.isneginf(lse[~some]).all()
    want = n[some].log()[:, None]
    off = (lse[some].double() - want).abs()
    assert (off <= 2.0 ** -22 * (want + 2)).all(), float(off.max())


CUT = [("bf16", 64, 32), ("fp16", 64, 64), ("fp16", 128, 32), ("bf16", 128, 128), ("bf16", 256, 64), ("fp16", 256, 128)]


@pytest.mark.parametrize("dtype,dim,group", CUT)
@pytest.mark.parametrize("batch,prefix,own", [(64, 3001, 300), (64, 6500, 40), (200, 1000, 700), (3, 6500, 500), (16, 1500, 3000)])
def test_prefix_of_single_tokens(awq, dtype, dim, group, batch, prefix, own):
    """On both paths, its items and units and the sequences' cut into pieces; sequences that end within it or are empty."""
    rng = np.random.default_rng(batch + prefix)
    lengths = [int(prefix + x) for x in rng.integers(1, own, batch)]
    lengths[0], lengths[-1] = prefix // 2, 0
    count_check(awq, dtype, dim, group, 2, 8 if batch > 8 else 4, 64, lengths, [1] * batch, prefix)


@pytest.mark.parametrize("dtype,dim,group", CUT)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("prefix", [0, 777, 5000])
def test_ragged_chunks(awq, dtype, dim, group, causal, prefix):
    """Chunks, drafts and single tokens, more rows than positions, with and without a prefix."""
    lengths = [prefix + 1700, prefix + 1, 0, max(50, prefix // 3), prefix + 900, 0, prefix + 60, prefix + 2005, prefix + 130]
    counts = [300, 1, 0, 53, 1, 40, 129, 5, 130]
    count_check(awq, dtype, dim, group, 2, 3, 16, lengths, counts, prefix, causal)


@pytest.mark.parametrize("dtype,dim,group", CUT)
@pytest.mark.parametrize("window,sinks", [(700, 33), (1, 1), (2048, 65), (300, 1000), (129, 0), (5000, 4)])
def test_windows_and_sinks(awq, dtype, dim, group, window, sinks):
    lengths = [6007, 1, 0, 90, 5200, 3000, 301, 64, 2049]
    counts = [400, 1, 0, 93, 1, 129, 5, 64, 1]
    count_check(awq, dtype, dim, group, 2, 3, 16, lengths, counts, window=window, sinks=sinks)
    count_check(awq, dtype, dim, group, 2, 8, 64, lengths, [1] * 9, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype,dim,group", CUT)
def test_whole_prompts(awq, dtype, dim, group):
    """More units than a line takes, and as many as it does."""
    count_check(awq, dtype, dim, group, 4, 8, 64, [2500, 2499], [2500, 2499])
    count_check(awq, dtype, dim, group, 4, 8, 64, [2500, 900], [900, 900], window=200, sinks=5)


@pytest.mark.parametrize("dtype,dim,group", CUT)
def test_prefix_beside_many_sequences(awq, dtype, dim, group):
    """The prefix's units a line by themselves."""
    counts = [1, 0, 2, 1, 3] * 14
    counts[7], counts[33] = 190, 71
    lengths = [int(2500 + n + 11 * i % 40) for i, n in enumerate(counts)]
    lengths[5], lengths[11] = 0, 700
    count_check(awq, dtype, dim, group, 8, 1, 16, lengths, counts, 2500, most=190)


@pytest.mark.parametrize("dim,group,dtype", [(64, 64, "fp16"), (128, 128, "bf16"), (256, 64, "fp16")])
@pytest.mark.parametrize("causal", [True, False])
def test_nan_in_a_prefix_and_beside_it_on_the_wide_path(awq, dim, group, dtype, causal):
    """It reaches the rows of its head that see it, and only those."""
    rng = np.random.default_rng(dim)
    heads, per, page, prefix, rows = 2, 4, 16, 128, 40
    lengths = [70, 170, 0, 128, 200]
    ptable, table, n_pages = with_prefix(rng, lengths, prefix, page)
    cache = filled(rng, n_pages, heads, dim, group, page)
    good = rng.standard_normal((heads, dim)).astype(np.float32)
    for pg, slot, head in ((ptable[6], 3, 1), (table[4, 11], 2, 0)):      # position 99, and 178 of the last sequence
        bad = good.copy()
        bad[head] = np.nan
        cache.write(pg, slot, bad, good)
    q = queries(rng, (len(lengths) * rows, heads * per, dim), dtype)
    say("NaN on the wide path", dim, causal)
    got, lse = attend(awq, q, dtype, cache, None, lengths, table, prefix=(ptable, prefix), causal=causal)
    check(q, dtype, cache, got, lse, None, lengths, table, prefix=(ptable, prefix), causal=causal)
    lost = torch.isnan(got).all(-1).view(len(lengths), rows, heads, per).all(-1).cpu()
    assert lost[1, :, 1].all() and not lost[0].any() and not lost[2].any() and not lost[1, :, 0].any()
    pos = torch.arange(160, 200)
    assert lost[4, :, 0].tolist() == ((pos >= 178) if causal else pos >= 0).tolist()
    assert lost[3, :, 1].tolist() == ((torch.arange(88, 128) >= 99) if causal else pos >= 0).tolist()


@pytest.mark.parametrize("view", [dict(prefix=333), dict(window=20, sinks=3)], ids=["prefix", "sinks"])
def test_tens_of_thousands_of_sequences(awq, view):
    rng = np.random.default_rng(2)
    lengths = [int(view.get("prefix", 0) + x) for x in rng.integers(1, 90, 1 << 16)]
    count_check(awq, "bf16", 64, 32, 4, 1, 16, lengths, [1] * len(lengths), **view)
    few = lengths[:1 << 13]
    count_check(awq, "fp16", 128, 64, 4, 1, 16, few, [1, 2, 0, 3] * (len(few) // 4), most=3, **view)
