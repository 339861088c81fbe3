"""Rules of the 4-bit key/value cache and its binding (CPU, no GPU)."""
from __future__ import annotations

import os

import numpy as np
import pytest

from oracle import kv_oracle as kv

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_quantization_awq_amd",
                   "libawq_mi355x.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run __graft_entry__.build())")


def test_rows_without_a_position():
    """Causal rows before position 0 see nothing; without causality every row sees the whole sequence."""
    rng = np.random.default_rng(0)
    c = kv.Cache(1, 1, 64, 64, 16)
    k, v = rng.standard_normal((2, 3, 1, 64)).astype(np.float32)
    kv.append(c, k, v, None, [3], np.array([[0]]))
    q = np.repeat(rng.standard_normal((1, 2, 64)), 5, 0)
    o, lse, _, _ = kv.attention(c, q, None, [3], np.array([[0]]))
    assert not o[:2].any() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
    o, lse, _, _ = kv.attention(c, q, None, [3], np.array([[0]]), causal=False)
    assert (o == o[-1:]).all() and (lse == lse[-1:]).all() and np.isfinite(lse).all()


@built
def test_a_cache_follows_its_pages():
    """The struct that calls hand to the library holds the pages' memory of that moment."""
    import torch
    from weight_only_quantization_awq_amd import awq
    pages = torch.zeros(4, 8, 2176, dtype=torch.uint8)
    c = awq.KvCache(pages, 128)
    struct, _ = awq._kv_pool(c)
    assert struct.pages == pages.data_ptr() and struct.n_pages == 4
    other = torch.zeros(6, 8, 2176, dtype=torch.uint8)
    pages.set_(other)
    struct, _ = awq._kv_pool(c)
    assert struct.pages == other.data_ptr() and struct.n_pages == 6
    pages.set_(other[2:])                                  # the same storage, further on
    assert awq._kv_pool(c)[0].pages == other[2].data_ptr() and awq._kv_pool(c)[0].n_pages == 4
    pages.resize_(40, 8, 2176)
    assert awq._kv_pool(c)[0].pages == pages.data_ptr() and awq._kv_pool(c)[0].n_pages == 40
    pages.set_(torch.zeros(4, 8, 2177, dtype=torch.uint8))
    with pytest.raises(ValueError):
        awq._kv_pool(c)


@built
@pytest.mark.parametrize("left", [0, 1, 4 * 8 * 2176 - 1])
def test_a_cache_without_its_memory_is_refused(left):
    import torch
    from weight_only_quantization_awq_amd import awq
    pages = torch.zeros(4, 8, 2176, dtype=torch.uint8)
    c = awq.KvCache(pages, 128)
    pages.untyped_storage().resize_(left)
    with pytest.raises(ValueError):
        awq._kv_pool(c)
    with pytest.raises(ValueError):
        awq.KvCache(pages, 128)


@built
def test_caches_can_be_looked_up():
    """The caches of a model's layers, in a list and as keys."""
    import torch
    from weight_only_quantization_awq_amd import awq
    layers = [awq.KvCache(torch.zeros(4, 8, 2176, dtype=torch.uint8), 128) for _ in range(3)]
    assert layers.index(layers[2]) == 2 and layers[0] != layers[1]
    assert {c: i for i, c in enumerate(layers)}[layers[1]] == 1
