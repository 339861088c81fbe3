"""The key/value quantiser's step is rounded to float32 and then to fp16: ranges whose product with
1/15 is a tie of fp16 only after the first of the two roundings (about one in 2^13) show it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv_oracle as kv

pytestmark = pytest.mark.gpu


def ranges(rng, n):
    """Ranges x with fp16(fl32(x/15)) != fp16(x/15), both with float32's 1/15."""
    found = np.empty(0, np.float32)
    fifteenth = np.float32(1) / np.float32(15)
    while len(found) < n:
        x = (rng.random(1 << 20) * 30 + 1).astype(np.float32)
        once = (x.astype(np.float64) * np.float64(fifteenth)).astype(np.float16)   # (48 bits: the product is exact)
        found = np.concatenate((found, x[(x * fifteenth).astype(np.float16) != once]))
    return found[:n]


def test_step_is_rounded_twice():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from weight_only_quantization_awq_amd import awq
    rng = np.random.default_rng(3)
    rows, heads, dim, group = 64, 2, 128, 32
    x = ranges(rng, 2 * rows * heads * dim // group).reshape(2, rows, heads, dim // group, 1)
    k, v = (x * rng.choice([0, 0.5, 1], (2, rows, heads, dim // group, group))).astype(np.float32).reshape(2, rows, heads, dim)
    k[..., ::group], v[..., ::group] = 0, 0
    k[..., 1::group], v[..., 1::group] = x[..., 0]
    table = rng.permutation(8)[None, :4]
    c = kv.Cache(8, heads, dim, group, 16)
    kv.append(c, k, v, None, [rows], table)
    dev = awq.kv_cache(8, heads, dim, group)
    awq.kv_append(dev, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), torch.tensor(table, dtype=torch.int32, device="cuda"),
                  torch.tensor([rows], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert np.array_equal(dev.pages.cpu().numpy(), c.bytes)
