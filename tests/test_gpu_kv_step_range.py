"""Queries of the rotated append where rows, weights and angles' factors are far from 1, in either direction, while
every value of the definition stays in float32's normal range.

Against 64 bits as in test_gpu_kv_step.py: u is off by 9 * 2^-24 of itself, then come the roundings of x*u, of the
weight's product, of a product with the cosine or sine, and of the sum: 13 * 2^-24 of M at most, which check_queries
writes as 16."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_kv import TYPES, ints
from tests.test_gpu_kv_step import angles, check_queries, dev, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (load anew: a test that reloads the module puts back a library that knows the classes of before)
    awq.load()
    return awq


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rot,interleaved", [("all", False), ("all", True), (16, False), (0, False)])
@pytest.mark.parametrize("size,heavy,turn", [(1e14, 1e25, 1.0), (1e-14, 1e-25, 1.0), (1e-14, 1e25, 1.0), (1e14, 1e-25, 1.0),
                                             (1e14, 1e20, 1e6), (1e-14, 1e-20, 1e-8), (1e18, 1e30, 1e3), (1e-18, 1e-28, 1e-3)])
def test_queries_over_the_range_of_float32(awq, dim, dtype, rot, interleaved, size, heavy, turn):
    rng = np.random.default_rng(dim)
    rot, rows, heads = dim if rot == "all" else rot, 5, 9
    q = (rng.standard_normal((rows, heads, dim)) * size).astype(np.float32)
    q[:, :, 0] = 3 * size                         # (no row whose mean is far from the others')
    q = torch.from_numpy(q).to(TYPES[dtype])
    w = (weight(rng, dim) * np.float32(heavy)).astype(np.float32)
    cs = (angles(rows, rot) * np.float32(turn)).astype(np.float32) if rot else None
    if cs is not None:
        cs[:, 1, :][cs[:, 1, :] == 0] = np.float32(turn) / 2      # (sines of position 0)
    k = torch.zeros(rows, 1, dim, dtype=TYPES[dtype], device="cuda")
    cache = awq.kv_cache(1, 1, dim, 64)
    say("range", dim, dtype, rot, interleaved, size, heavy, turn)
    out = awq.kv_append_rotated(cache, q.cuda(), k, k, ints([[0]]), ints([rows]), dev(cs), q_weight=dev(w), eps=1e-45,
                                interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    check_queries(out, q.float().numpy(), w, cs, np.arange(rows), 1e-45, interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_small_channels_beside_large_ones(awq, dtype, interleaved):
    """One channel pair of 2^-90 in a row of 2^-40, with weights of 2^30: results of 2^-20."""
    dim, rows = 128, 3
    rng = np.random.default_rng(1)
    q = rng.standard_normal((rows, 4, dim)).astype(np.float32) * np.float32(2.0 ** -40)
    pair = (6, 7) if interleaved else (6, 6 + dim // 2)
    q[..., pair] = (1 + rng.random((rows, 4, 2)).astype(np.float32)) * np.float32(2.0 ** -90)
    q = torch.from_numpy(q).to(TYPES[dtype])
    w = np.full(dim, 2.0 ** -40, np.float32)
    w[list(pair)] = 2.0 ** 30
    cs = angles(rows, dim)
    k = torch.zeros(rows, 1, dim, dtype=TYPES[dtype], device="cuda")
    say("small channels", dtype, interleaved)
    out = awq.kv_append_rotated(awq.kv_cache(1, 1, dim, 64), q.cuda(), k, k, ints([[0]]), ints([rows]), dev(cs), q_weight=dev(w),
                                eps=1e-45, interleaved=interleaved)
    torch.cuda.synchronize()
    check_queries(out, q.float().numpy(), w, cs, np.arange(rows), 1e-45, interleaved)
