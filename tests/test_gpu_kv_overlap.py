"""The rotated append writing its queries where keys or values lie, and attention its output where its queries lie:
as with tensors of their own, bit for bit."""
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


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("view", ["plain", "sinks", "prefix"])
def test_attention_in_place(awq, dim, group, view):
    """Items and units whole and cut into pieces, on both paths, in slices of a fused projection."""
    rng = np.random.default_rng(dim)
    torch.manual_seed(dim)
    heads, per, page = 2, 4, 16
    lengths, counts = [3000, 17, 700, 90, 0, 2500], [300, 1, 40, 2, 1, 1]
    table, n_pages = table_for(lengths, page, rng)
    cache = awq.kv_cache(n_pages, heads, dim, group, page)
    k, v = (torch.randn(sum(lengths), heads, dim, device="cuda").bfloat16() for _ in range(2))
    t, n = ints(table), ints(lengths)
    awq.kv_append(cache, k, v, t, n, row_start=ints(np.concatenate(([0], np.cumsum(lengths)))))
    start = np.concatenate(([0], np.cumsum(counts)))
    kw = dict(window=400, sinks=20) if view == "sinks" else dict(prefix=(t[0].clone(), ints([1000]))) if view == "prefix" else {}
    x = torch.randn(sum(counts), heads * per + 3, dim, device="cuda").bfloat16()
    for most in (300, 2):       # (2: the long ones are left as they were, without a prefix)
        rows = list(range(sum(counts))) if most == 300 else [300, 341, 342, 343, 344]
        q = x.clone()[:, 1:-2]
        say("attention in place", dim, view, most)
        want, want_lse = awq.kv_attention(q, cache, t, n, row_start=ints(start), max_rows=most, want_lse=True, out=torch.zeros_like(q), **kw)
        got, lse = awq.kv_attention(q, cache, t, n, row_start=ints(start), max_rows=most, want_lse=True, out=q, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got[rows], want[rows]) and torch.equal(lse[rows], want_lse[rows])
    with pytest.raises(awq.AwqError, match="share memory"):
        awq.kv_attention(x[:, :-3], cache, t, n, row_start=ints(start), out=x[:, 1:-2], **kw)
