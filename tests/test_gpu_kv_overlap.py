"""The rotated append writing its queries where keys or values lie: as with tensors of their own, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_kv import ints, table_for
from tests.test_gpu_kv_step import angles, dev, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (load anew: a test that reloads the module puts back a library that knows the classes of before)
    awq.load()
    return awq


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("where", ["K", "V", "between", "Q and K", "rows of another stride"])
@pytest.mark.parametrize("rows,batch,ragged", [(1, 1, False), (7, 7, False), (3000, 3, True)])
def test_queries_over_keys_and_values(awq, dim, where, rows, batch, ragged):
    rng = np.random.default_rng(dim + rows)
    torch.manual_seed(dim + rows)
    heads = 4
    counts = [rows // batch] * batch
    if ragged:
        counts[0], counts[1] = counts[0] - 300, counts[1] + 300
    lengths = [n + int(rng.integers(0, 40)) for n in counts]
    table, n_pages = table_for(lengths, 16, rng)
    start = ints(np.concatenate(([0], np.cumsum(counts)))) if ragged else None
    cs, w = dev(angles(max(lengths), dim)), dev(weight(rng, dim))
    q = torch.randn(rows, heads, dim, device="cuda").bfloat16()
    both = torch.randn(rows, 2 * heads, dim, device="cuda").bfloat16()       # keys and values of a fused projection
    k, v, out = both[:, :heads], both[:, heads:], None
    if where == "K":
        out = k
    elif where == "V":
        out = v
    elif where == "between":
        out = both[:, heads // 2:heads // 2 + heads]
    elif where == "Q and K":                                                 # in place, of queries that are the keys
        q = out = k
    else:
        v = v.contiguous()
        k = k.contiguous()
        room = torch.zeros(3 * rows + 2, heads, dim, dtype=torch.bfloat16, device="cuda")
        room[rows:2 * rows].copy_(k)
        k, out = room[rows:2 * rows], room[:2 * rows].view(rows, 2 * heads, dim)[:, 1:heads + 1]
    args = (ints(table), ints(lengths), cs)
    kw = dict(row_start=start, q_weight=w, k_weight=w)
    apart, shared = awq.kv_cache(n_pages, heads, dim, 64), awq.kv_cache(n_pages, heads, dim, 64)
    say("queries over", where, dim, rows)
    want = awq.kv_append_rotated(apart, q.clone(), k.clone(), v.clone(), *args, **kw)
    got = awq.kv_append_rotated(shared, q, k, v, *args, out=out, **kw)
    torch.cuda.synchronize()
    assert got is out and torch.equal(got, want) and torch.equal(shared.pages, apart.pages)


def test_bindings_refuse_an_output_over_other_queries(awq):
    q = torch.zeros(4, 9, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    cache, args = awq.kv_cache(4, 2, 64, 64), (ints([[0], [1], [2], [3]]), ints([1, 1, 1, 1]), None)
    with pytest.raises(awq.AwqError, match="share memory"):
        awq.kv_append_rotated(cache, q[:, :8], k, k, *args, out=q[:, 1:])
    with pytest.raises(awq.AwqError, match="share memory"):
        awq.kv_append_rotated(cache, q[:2], k[:2], k[:2], ints([[0], [1]]), ints([1, 1]), None, out=q[1:3])
    awq.kv_append_rotated(cache, q[:2], k[:2], k[:2], ints([[0], [1]]), ints([1, 1]), None, out=q[2:])
    torch.cuda.synchronize()
