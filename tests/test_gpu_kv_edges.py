"""The 4-bit key/value cache on the GPU, at the ends of what its calls allow: more rows than
announced, weights far below the largest, pools and slots that nothing was written to.
Tolerances of attention as derived in test_gpu_kv.py, unless a test derives its own."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv_oracle as kv
from tests import test_gpu_kv as base
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (as in test_gpu_kv.py)
    awq.load()
    return awq


@pytest.mark.parametrize("dim,per,max_rows", [(128, 1, 1), (64, 1, 3), (128, 3, 1), (256, 8, 1), (64, 40, 1)])
def test_more_rows_than_max_rows(awq, dim, per, max_rows):
    """Sequences with more rows than max_rows, just above it and far above, next to others: theirs
    alone are unspecified, and nothing outside O, lse and the workspace is written."""
    rng = np.random.default_rng(dim + per + max_rows)
    heads, group, page = 2, 64, 16
    over = [max_rows + 1, max(max_rows + 1, 16 // per), 100]
    lengths = [2000, 700, 31, 1500, 900, 1, 1200]
    counts = [over[1], max_rows, 1, over[0], max_rows, 1, over[2]]
    table, n_pages = base.table_for(lengths, page, rng)
    cache = base.filled(rng, n_pages, heads, dim, group, page)
    base.spoil(cache, table, lengths)
    start = np.concatenate(([0], np.cumsum(counts)))
    last = int(start[-1])
    q = base.queries(rng, (last + 5, heads * per, dim), "fp16")
    qd = torch.from_numpy(q).half().cuda()
    dev = base.pool(awq, cache)
    size = awq.kv_attention_workspace_size(dev, heads * per, len(q), len(lengths), table.shape[1], True, max_rows)
    assert size > 0
    guard = 1 << 16
    room = torch.full((size + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((len(q) + 8, heads * per, dim), 7.0, dtype=torch.float16, device="cuda")
    say("max_rows", dim, per, max_rows)
    got, lse = awq.kv_attention(qd, dev, base.ints(table), base.ints(lengths), row_start=base.ints(start), max_rows=max_rows,
                                out=out[:len(q)], workspace=room[:size], want_lse=True)
    torch.cuda.synchronize()
    assert (room[size:] == 0xA5).all()
    assert (out[last:] == 7.0).all()
    keep = [b for b, n in enumerate(counts) if n <= max_rows]
    rows = np.concatenate([np.arange(start[b], start[b + 1]) for b in keep])
    some = np.concatenate(([0], np.cumsum([counts[b] for b in keep])))
    base.check(q[rows], "fp16", cache, got[rows.tolist()], lse[rows.tolist()], some, [lengths[b] for b in keep], table[keep])
