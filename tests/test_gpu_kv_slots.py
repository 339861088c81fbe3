"""Slots of a step on pages at and behind the pool's end: none, where the call is told the pool's size, and none that
the cache's other calls do not use."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv_step_oracle as step
from tests.gpu_util import say
from tests.test_gpu_kv import ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (load anew: a test that reloads the module puts back a library that knows the classes of before)
    awq.load()
    return awq


@pytest.mark.parametrize("n_pages", [1, 40, 41, (1 << 31) - 1])
@pytest.mark.parametrize("given", [False, True])
def test_slots_end_with_the_pool(awq, n_pages, given):
    """Pages of either kind, in the table and handed out: n_pages - 1, n_pages, beyond, and the largest number."""
    rng = np.random.default_rng(n_pages % 1000)
    page, batch, most, top = 16, 50, 6, (1 << 31) - 1
    pick = np.array([0, n_pages - 1, min(n_pages, top), min(n_pages + 1, top), top, -1, -(1 << 31)])
    table, free = rng.choice(pick, (batch, most)), rng.choice(pick, 400)
    kv_len, count = rng.integers(0, 40, batch), rng.integers(0, 56, batch)
    rows = int(count.sum()) + 3
    want = step.tables(page, kv_len, count, free, 2, table, rows)
    slots = np.where(want[5] // page < n_pages, want[5], -1)
    out = None
    if given:
        i32 = dict(dtype=torch.int32, device="cuda")
        out = awq.KvStep(torch.empty(batch, **i32), torch.empty(batch + 1, **i32), torch.empty(1, **i32), torch.empty(rows, **i32),
                         torch.empty(rows, dtype=torch.int64, device="cuda"))
    dev = ints(table)
    say("slots", n_pages, given)
    got = awq.kv_tables(dev, ints(kv_len), ints(count), ints(free), ints([2]), page=page, rows=rows, out=out, n_pages=n_pages)
    torch.cuda.synchronize()
    assert np.array_equal(got.slot.cpu().numpy(), slots) and (n_pages == top or (slots != want[5]).any())
    # all else is as it is without
    for x, y in zip((dev, got.kv_len, got.row_start, got.taken, got.position), want):
        assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(y).reshape(-1))
    plain = awq.kv_tables(ints(table), ints(kv_len), ints(count), ints(free), ints([2]), page=page, rows=rows)
    assert np.array_equal(plain.slot.cpu().numpy(), want[5])


def test_a_step_has_the_slots_that_append_writes(awq):
    """Tokens appear in the pool at the step's slots, and nowhere else."""
    page, dim, heads, n_pages = 16, 64, 2, 6
    cache = awq.kv_cache(n_pages, heads, dim, 64, page)
    table, free = ints([[3, -1, -1], [6, -1, -1], [1, -1, -1]]), ints([2, 7, 5, 6, 0])      # 6 and 7 are not in the pool
    count = [20, 4, 18]
    s = awq.kv_tables(table, ints([10, 7, 16]), ints(count), free, page=page, rows=sum(count), n_pages=n_pages)
    x = torch.full((sum(count), heads, dim), 3.0, device="cuda")
    say("slots of an append")
    awq.kv_append(cache, x, x, table, s.kv_len, row_start=s.row_start)
    every = ints(np.arange(n_pages).reshape(1, -1))
    k, _ = awq.kv_read(cache, every, ints([n_pages * page]), n_pages * page, dtype=torch.float32)
    written = torch.nonzero(k[:, 0, 0] == 3.0)[:, 0].tolist()
    slots = s.slot.tolist()
    assert sorted(y for y in slots if y >= 0) == written and slots.count(-1) > 4
    with pytest.raises(awq.AwqError, match="n_pages"):
        awq.kv_tables(table, s.kv_len, s.kv_len, free, page=page, n_pages=-1)


@pytest.mark.parametrize("batch,rows", [(1 << 21, 5000), (1 << 20, 1 << 21), (100003, 77)])
def test_tables_of_the_largest_batches(awq, batch, rows):
    """The definitions for all sequences at once; half of the pages that they need, some behind the pool's end."""
    rng = np.random.default_rng(rows)
    page, most, n_pages = 16, 4, 900
    kv_len, count = rng.integers(0, 50, batch), rng.integers(0, 3, batch)
    count[rng.integers(0, batch, 50)] = 1000
    n = np.clip(count, 0, page * most - kv_len)
    now, have = kv_len + n, -(-kv_len // page)
    need = -(-now // page) - have
    free, table = rng.integers(0, 1000, int(need.sum()) // 2), rng.integers(0, 1000, (batch, most))
    dev = ints(table)
    say("tables", batch, rows)
    got = awq.kv_tables(dev, ints(kv_len), ints(count), ints(free), page=page, rows=rows, n_pages=n_pages)
    torch.cuda.synchronize()
    j = np.arange(most) - have[:, None]
    which = (np.cumsum(need) - need)[:, None] + j
    want = np.where((j >= 0) & (j < need[:, None]), np.where(which < len(free), free[np.clip(which, 0, len(free) - 1)], -1), table)
    start = np.concatenate(([0], np.cumsum(n)))
    r = np.arange(rows)
    b = np.minimum(np.searchsorted(start[1:], r, side="right"), batch - 1)
    position = np.where(r < start[-1], kv_len[b] + r - start[b], -1)
    pg = want[b, np.maximum(position, 0) // page]
    slot = np.where((position >= 0) & (pg >= 0) & (pg < n_pages), pg * page + position % page, -1)
    for name, x, y in (("table", dev, want), ("kv_len", got.kv_len, now), ("row_start", got.row_start, start),
                       ("taken", got.taken, [need.sum()]), ("position", got.position, position), ("slot", got.slot, slot)):
        assert np.array_equal(x.cpu().numpy(), y), name
