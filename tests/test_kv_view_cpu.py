"""Sinks and shared prefixes without a GPU: the oracle by hand, the view's layout, workspace sizes
and the arguments that validation refuses (before any HIP call)."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import kv_oracle as kv
from oracle import kv_step_oracle as step
from tests.test_kv_step_cpu import ARG, FAKE, LIB, ROOT, SHAPE, _batch, _cache

built = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run __graft_entry__.build())")
WORKSPACE = -4


# ---- the oracle -------------------------------------------------------------

def test_what_a_row_sees_by_hand():
    t = np.arange(12)
    assert t[step.sees(9, t, True, 3, 2)].tolist() == [0, 1, 7, 8, 9]
    assert t[step.sees(1, t, True, 3, 5)].tolist() == [0, 1]
    assert t[step.sees(9, t, True, 3, 8)].tolist() == list(range(10))
    assert t[step.sees(4, t, False, 0, 0)].tolist() == t.tolist()


def test_a_view_of_nothing_is_attention():
    rng = np.random.default_rng(0)
    c = kv.Cache(4, 2, 64, 32, 16)
    k, v = rng.standard_normal((2, 40, 2, 64)).astype(np.float32)
    table = np.array([[2, 0, 3]])
    kv.append(c, k, v, None, [40], table)
    q = rng.standard_normal((5, 4, 64))
    for a, b in zip(step.attention(c, q, None, [40], table, window=9), kv.attention(c, q, None, [40], table, window=9)):
        assert np.array_equal(a, b)
    # a prefix that lies where the table says
    for a, b in zip(step.attention(c, q, None, [40], np.array([[-1, 0, 3]]), prefix=([2], 16)), kv.attention(c, q, None, [40], table)):
        assert np.array_equal(a, b)


# ---- the library ------------------------------------------------------------

@pytest.fixture(scope="module")
def awq():
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (load anew: a test that reloads the module puts back a library that knows the classes of before)
    return awq


@built
def test_struct_layout_matches_the_header(awq, tmp_path):
    src = tmp_path / "sizes.c"
    t = awq._KvViewC
    lines = 'printf("%zu ", sizeof(awq_kv_view));' + "".join(f'printf("%zu ", offsetof(awq_kv_view, {f[0]}));' for f in t._fields_)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "awq.h"\nint main(void) {' + lines + "}\n")
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]


def _call(awq, cache=None, batch=None, view=True, q=FAKE, t=1, q_heads=8, q_stride=1024, max_rows=2, scale=1.0, causal=1, out=FAKE,
          out_stride=1024, lse=None, ws=FAKE, ws_bytes=1 << 40, **over):
    v = awq._KvViewC(**{**dict(window=0, sinks=0, prefix_table=None, prefix_len=None, prefix_pages=0), **over})
    return awq.load().awq_kv_attention_ex(_cache(awq) if cache is None else cache, _batch(awq) if batch is None else batch,
                                          v if view else None, q, t, q_heads, q_stride, max_rows, scale, causal, out, out_stride, lse,
                                          ws, ws_bytes, None)


PREFIX = dict(prefix_table=FAKE, prefix_len=FAKE, prefix_pages=3)
BAD = [(dict(view=False), ARG), (dict(window=-1), ARG), (dict(sinks=-1, window=5), ARG), (dict(sinks=1), ARG),
       (dict(sinks=1, window=5, causal=0), ARG), (dict(window=5, **PREFIX), ARG), (dict(sinks=5, **PREFIX), ARG),
       (dict(sinks=5, window=5, **PREFIX), ARG),
       (dict(PREFIX, prefix_table=None), ARG), (dict(PREFIX, prefix_table=FAKE + 2), ARG), (dict(PREFIX, prefix_len=FAKE + 1), ARG),
       (dict(PREFIX, prefix_pages=0), SHAPE), (dict(PREFIX, prefix_pages=-1), SHAPE), (dict(PREFIX, prefix_pages=1 << 28), SHAPE),
       (dict(PREFIX, prefix_pages=1 << 62), SHAPE), (dict(PREFIX, ws=None), WORKSPACE), (dict(PREFIX, ws=FAKE + 8), WORKSPACE),
       (dict(PREFIX, ws_bytes=2 * 6 * 8 * 130 * 4 - 1), WORKSPACE), (dict(PREFIX, q_heads=7), SHAPE), (dict(PREFIX, scale=0.0), ARG),
       (dict(PREFIX, lse=FAKE + 2), ARG), (dict(window=5, sinks=2, t=0), -3)]


@built
@pytest.mark.parametrize("over,want", BAD)
def test_attention_refuses(awq, over, want):
    assert _call(awq, **over) == want
    assert awq.load().awq_last_error() != b""


@built
def test_a_prefix_of_too_many_rows_is_refused(awq):
    """dim/4 threads to a row and query head of the join: fewer than 2^32."""
    over = dict(q_heads=128, q_stride=16384, out_stride=16384, cache=_cache(awq, heads=1), max_rows=1)
    for rows, want in ((1 << 20, SHAPE), ((1 << 20) - 1024, WORKSPACE)):
        b = _batch(awq, rows=rows, batch=1024)
        assert _call(awq, batch=b, ws_bytes=0, **PREFIX, **over) == want


@built
def test_no_rows_need_nothing(awq):
    none = _batch(awq, rows=0)
    assert _call(awq, batch=none, q=None, out=None, window=5, sinks=1, ws=None, ws_bytes=0) == 0
    assert _call(awq, batch=none, q=None, out=None, **PREFIX) == 0


@built
def test_workspace_sizes(awq):
    """Sinks need what the call without them does; a prefix adds the sums of every row and query head, its own and
    the prefix's, dim + 2 floats each, and at most what the prefix alone would need."""
    lib = awq.load()
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    for dim, q_heads, rows, most, ragged in ((128, 8, 6, 40, False), (64, 64, 96, 300, True), (256, 4, 3000, 7, True)):
        c = _cache(awq, dim=dim, group=64, page_stride=1 << 20)
        b = _batch(awq, rows=rows, max_pages=most, row_start=FAKE if ragged else None)
        size = lambda **v: lib.awq_kv_attention_workspace_size_ex(  # noqa: E731
            c, b, awq._KvViewC(**{**dict(window=0, sinks=0, prefix_table=None, prefix_len=None, prefix_pages=0), **v}), q_heads, 0)
        plain = lib.awq_kv_attention_workspace_size(c, b, q_heads, 0)
        assert size() == size(window=9, sinks=3) == plain
        sums = 2 * (up(rows * q_heads * 8) + up(rows * q_heads * dim * 4))
        last = 0
        for pages in (1, 50, 5000):
            n = size(prefix_len=FAKE, prefix_pages=pages)
            assert n >= sums and n >= last
            last = n
    assert size(prefix_len=FAKE, prefix_pages=0) == 0 and lib.awq_last_error() != b""


@built
def test_binding_sizes(awq):
    import torch
    c = awq.KvCache(torch.zeros(4, 2, 16 * 64 + 8 * 16, dtype=torch.uint8), 64, 64, 16)
    assert awq.kv_attention_workspace_size(c, 8, 12, 3, 100, prefix_pages=1) >= 2 * 12 * 8 * 66 * 4
    with pytest.raises(awq.AwqError):
        awq.kv_attention_workspace_size(c, 8, 12, 3, 100, prefix_pages=-1)
