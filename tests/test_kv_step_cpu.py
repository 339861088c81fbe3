"""A step's tables and the rotated append without a GPU: the oracle by hand, struct layouts and
the arguments that validation refuses (before any HIP call)."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import kv_oracle as kv
from oracle import kv_step_oracle as step

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "weight_only_quantization_awq_amd", "libawq_mi355x.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run __graft_entry__.build())")

FAKE = 0x10000  # never dereferenced: validation fails before any HIP call
ARG, SHAPE, DTYPE = -1, -2, -3


# ---- the oracle -------------------------------------------------------------

def test_tables_by_hand():
    table = [[7, -1, -1], [8, 9, -1], [-1, -1, -1], [5, 6, 4]]
    got = step.tables(16, [15, 32, 0, 47], [2, 1, 0, 9], [20, 21, 22], 1, table, 6)
    assert got[0].tolist() == [[7, 21, -1], [8, 9, 22], [-1, -1, -1], [5, 6, 4]]
    assert got[1].tolist() == [17, 33, 0, 48]           # the last sequence takes one row, not nine
    assert got[2].tolist() == [0, 2, 3, 3, 4] and got[3] == 3
    assert got[4].tolist() == [15, 16, 32, 47, -1, -1]
    assert got[5].tolist() == [7 * 16 + 15, 21 * 16, 22 * 16, 4 * 16 + 15, -1, -1]


def test_tables_without_pages_left():
    got = step.tables(16, [0, 16], [17, 1], [3], 0, [[-1, -1], [9, -1]], 18)
    assert got[0].tolist() == [[3, -1], [9, -1]] and got[3] == 3
    assert got[5][15] == 63 and got[5][16] == -1 and got[5][17] == -1 and got[4][17] == 16


def test_rotation_by_hand():
    """A quarter turn of position 1; halves pair i with i + rot/2, neighbours 2i with 2i + 1."""
    cs = np.zeros((2, 2, 8), np.float32)
    cs[0, 0] = 1
    cs[1, 1] = 1
    x = np.arange(64, dtype=np.float32)[None, None]
    y = step.turned(x, None, cs, np.array([1]))
    assert y[0, 0, :8].tolist() == [-8.0 - i for i in range(8)] and y[0, 0, 8:16].tolist() == list(range(8))
    assert (y[0, 0, 16:] == x[0, 0, 16:]).all()
    y = step.turned(x, None, cs, np.array([1]), interleaved=True)
    assert y[0, 0, :6].tolist() == [-1, 0, -3, 2, -5, 4]
    assert (step.turned(x, None, cs, np.array([0])) == x).all()
    assert np.isnan(step.turned(x, None, cs, np.array([2]))).all()


def test_norm_by_hand():
    x = np.full((1, 1, 64), -3.0, np.float32)
    y = step.turned(x, np.arange(64, dtype=np.float32), None, np.array([0]), eps=7.0)   # sqrt(9 + 7) = 4
    assert (y[0, 0] == np.float32(-0.75) * np.arange(64)).all()


def test_rotation_keeps_products_of_equal_distance():
    """q at p and k at p - d: the product depends on d alone."""
    from math import pi
    freq = 10000.0 ** (-np.arange(32) / 32)
    angle = np.arange(50)[:, None] * freq
    cs = np.stack((np.cos(angle), np.sin(angle)), 1).astype(np.float32)
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 64)).astype(np.float32)
    for inter in (False, True):
        dots = [(step.turned(q, None, cs, np.array([p]), interleaved=inter).astype(np.float64)
                 * step.turned(k, None, cs, np.array([p - 5]), interleaved=inter)).sum() for p in (5, 17, 49)]
        # angles of up to 49 in float32's cosines (2^-24 each), products of 3 roundings
        assert np.ptp(dots) <= 64 * 8 * 2.0 ** -24 * np.abs(q).max() * np.abs(k).max() * pi


def test_append_rotated_of_nothing_is_append():
    rng = np.random.default_rng(1)
    a, b = (kv.Cache(2, 2, 64, 32, 16) for _ in range(2))
    q, k, v = rng.standard_normal((3, 5, 2, 64)).astype(np.float32)
    out = step.append_rotated(a, q, k, v, None, [7], np.array([[1]]), None)
    kv.append(b, k, v, None, [7], np.array([[1]]))
    assert (a.bytes == b.bytes).all() and (out == q).all()


# ---- the library ------------------------------------------------------------

@pytest.fixture(scope="module")
def awq():
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (load anew: a test that reloads the module puts back a library that knows the classes of before)
    return awq


@built
def test_struct_layouts_match_the_header(awq, tmp_path):
    src = tmp_path / "sizes.c"
    names = {"awq_kv_rotation": awq._KvRotationC, "awq_kv_step": awq._KvStepC}
    lines = [f'printf("%zu ", sizeof({n}));' + "".join(f'printf("%zu ", offsetof({n}, {f[0]}));' for f in t._fields_)
             for n, t in names.items()]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "awq.h"\nint main(void) {' + "".join(lines) + "}\n")
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    want = []
    for t in names.values():
        want += [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]
    assert got == want


def _cache(awq, **over):
    return awq._KvCacheC(**{**dict(pages=FAKE, n_pages=8, page_stride=4 * 16 * 136, heads=4, dim=128, group=128, page=16), **over})


def _batch(awq, **over):
    return awq._KvBatchC(**{**dict(rows=6, batch=3, max_pages=4, row_start=None, kv_len=FAKE, block_table=FAKE), **over})


def _rotated(awq, cache=None, batch=None, rotation=None, q=FAKE, k=FAKE, v=FAKE, t=1, q_heads=8, q_stride=1024, k_stride=512,
             v_stride=512, out=2 * FAKE, out_stride=1024, **rot):
    r = awq._KvRotationC(**{**dict(cos_sin=FAKE, positions=64, rot=128, interleaved=0, q_weight=FAKE, k_weight=FAKE, eps=1e-6), **rot})
    return awq.load().awq_kv_append_rotated(_cache(awq) if cache is None else cache, _batch(awq) if batch is None else batch,
                                            r if rotation is None else rotation, q, k, v, t, q_heads, q_stride, k_stride, v_stride,
                                            out, out_stride, None)


BAD_ROTATED = [
    (dict(rot=-16), SHAPE), (dict(rot=144), SHAPE), (dict(rot=8), SHAPE), (dict(rot=24), SHAPE), (dict(interleaved=2), ARG),
    (dict(interleaved=-1), ARG), (dict(positions=0), SHAPE), (dict(positions=-1), SHAPE), (dict(positions=(1 << 30) + 1), SHAPE),
    (dict(cos_sin=None), ARG), (dict(cos_sin=FAKE + 4), ARG), (dict(q_weight=FAKE + 4), ARG), (dict(k_weight=FAKE + 8), ARG),
    (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(t=3), DTYPE), (dict(t=-1), DTYPE), (dict(q_heads=0), SHAPE), (dict(q_heads=65536), SHAPE), (dict(q_stride=1016), SHAPE),
    (dict(q_stride=1028), SHAPE), (dict(out_stride=512), SHAPE), (dict(q=None), ARG), (dict(q=FAKE + 2), ARG), (dict(out=None), ARG),
    (dict(k=None), ARG), (dict(v=FAKE + 8), ARG), (dict(k_stride=511), SHAPE), (dict(out=FAKE, out_stride=2048), ARG),
]


@built
@pytest.mark.parametrize("over,want", BAD_ROTATED)
def test_append_rotated_refuses(awq, over, want):
    assert _rotated(awq, **over) == want
    assert awq.load().awq_last_error() != b""


@built
def test_append_rotated_refuses_structs_and_sizes(awq):
    null = ctypes.POINTER(awq._KvRotationC)()
    assert _rotated(awq, rotation=null) == ARG
    assert _rotated(awq, batch=_batch(awq, rows=7)) == SHAPE
    assert _rotated(awq, cache=_cache(awq, dim=96)) == SHAPE
    many = _batch(awq, rows=1 << 23, batch=1 << 20, max_pages=1)
    assert _rotated(awq, cache=_cache(awq, heads=1), batch=many, q_heads=1024, q_stride=1 << 17, out_stride=1 << 17) == SHAPE
    # as many threads for queries as for keys, 2^32 together
    many = _batch(awq, rows=1 << 25, batch=1, max_pages=1)
    assert _rotated(awq, cache=_cache(awq, heads=1), batch=many, q_heads=1) == SHAPE
    assert b"q_heads" in awq.load().awq_last_error()
    assert _rotated(awq, batch=_batch(awq, rows=0), q=None, k=None, v=None, out=None) == 0
    # nothing rotated and no norm: no table, no eps
    assert _rotated(awq, batch=_batch(awq, rows=0), rot=0, positions=0, cos_sin=None, q_weight=None, k_weight=None, eps=0.0) == 0


def _tables(awq, page=16, batch=3, max_pages=4, kv_len=0x1000, count=0x2000, free=0x3000, n_free=5, taken=0x4000, table=0x5000,
            rows=7, step=True, **over):
    s = awq._KvStepC(**{**dict(kv_len=0x6000, row_start=0x7000, taken=0x8000, position=0x9000, slot=0xA000), **over})
    return awq.load().awq_kv_tables(page, batch, max_pages, kv_len, count, free, n_free, taken, table, rows,
                                    s if step else None, None)


BAD_TABLES = [
    (dict(page=0), ARG), (dict(page=24), ARG), (dict(page=512), ARG), (dict(batch=0), SHAPE), (dict(batch=(1 << 21) + 1), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 27), SHAPE), (dict(max_pages=1 << 62), SHAPE), (dict(rows=-1), SHAPE),
    (dict(rows=(1 << 30) + 1), SHAPE), (dict(n_free=-1), SHAPE), (dict(n_free=1 << 31), SHAPE), (dict(kv_len=None), ARG),
    (dict(count=None), ARG), (dict(free=None), ARG), (dict(table=None), ARG), (dict(step=False), ARG), (dict(row_start=None), ARG),
    (dict(kv_len=0x1002), ARG), (dict(slot=0xA004), ARG), (dict(position=0x9001), ARG), (dict(table=0x5002), ARG),
    (dict(taken=0x4002), ARG),
]


@built
@pytest.mark.parametrize("over,want", BAD_TABLES)
def test_tables_refuse(awq, over, want):
    assert _tables(awq, **over) == want
    assert awq.load().awq_last_error() != b""


@built
@pytest.mark.parametrize("name", ["kv_len", "row_start", "taken", "position", "slot"])
@pytest.mark.parametrize("at", [0x1000, 0x2000, 0x3000, 0x4000])
def test_tables_refuse_outputs_that_are_inputs(awq, name, at):
    s = dict(kv_len=0x6000, row_start=0x7000, taken=0x8000, position=0x9000, slot=0xA000)
    c = awq._KvStepC(**{**s, name: at})
    assert awq.load().awq_kv_tables(16, 3, 4, 0x1000, 0x2000, 0x3000, 5, 0x4000, 0x5000, 7, c, None) == ARG
    assert b"input" in awq.load().awq_last_error()


@built
@pytest.mark.parametrize("over", [dict(kv_len=0x1008), dict(row_start=0x1FF4), dict(position=0x2FE8), dict(slot=0x3010), dict(kv_len=0x3FF8),
                                  dict(row_start=0x5FFC - 8), dict(position=0x6008), dict(slot=0x7008), dict(taken=0x502C),
                                  dict(position=0x8000 - 24)])
def test_tables_refuse_shared_memory(awq, over):
    """3 sequences, 4 pages each, 5 free pages, 7 rows: arrays that begin elsewhere and still share an element."""
    c = awq._KvStepC(**{**dict(kv_len=0x6000, row_start=0x7000, taken=0x8000, position=0x9000, slot=0xA000), **over})
    assert awq.load().awq_kv_tables(16, 3, 4, 0x1000, 0x2000, 0x3000, 5, 0x4000, 0x5000, 7, c, None) == ARG
    assert b"share memory" in awq.load().awq_last_error()


@built
def test_binding_refuses_cpu_tensors_and_types(awq):
    import torch
    pages = torch.zeros(4, 2, 16 * 64 + 8 * 16, dtype=torch.uint8)
    c = awq.KvCache(pages, 64, 64, 16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    x = torch.zeros(1, 2, 64)
    with pytest.raises(ValueError):
        awq.kv_append_rotated(c, x, x, x, i, i[0], None)
    with pytest.raises(TypeError):
        awq.kv_append_rotated(c, x, x.half(), x, i, i[0], None)
    with pytest.raises(ValueError):
        awq.kv_tables(i, i[0], i[0], i[0])


@built
def test_rotation_table(awq):
    t = awq.kv_rotation_table(4000, 64, base=500.0, device="cpu").numpy()
    assert t.shape == (4000, 2, 32) and t.dtype == np.float32
    angle = np.arange(4000)[:, None] * 500.0 ** (-np.arange(0, 64, 2) / 64)
    # an angle in float64 is off by 4000 * 2^-52, a value rounded once to float32
    assert np.abs(t - np.stack((np.cos(angle), np.sin(angle)), 1)).max() <= 2.0 ** -25 + 4000 * 2.0 ** -50
