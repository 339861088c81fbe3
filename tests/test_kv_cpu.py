"""The 4-bit key/value cache without a GPU: the oracle's own checks, page sizes,
workspace sizes and the arguments that validation refuses (before any HIP call)."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import kv_oracle as kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "weight_only_quantization_awq_amd", "libawq_mi355x.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run __graft_entry__.build())")

FAKE = 0x10000  # never dereferenced: validation fails before any HIP call
ARG, SHAPE, DTYPE, WORKSPACE = -1, -2, -3, -4


# ---- the oracle -------------------------------------------------------------

@pytest.mark.parametrize("dim,group,page", [(64, 32, 16), (64, 64, 32), (128, 128, 16), (256, 64, 64)])
def test_layout_uses_every_nibble_once(dim, group, page):
    seen = set()
    for t in range(page):
        for c in range(dim):
            for at, shift in (kv.key_place(dim, t, c), kv.value_place(page, dim, t, c)):
                assert 0 <= at < page * dim
                seen.add((at, shift))
    assert len(seen) == 2 * page * dim


def test_key_words_hold_the_pack_order():
    """Word kb*J + j of a token is the packed word of channels 32j + 8kb + 0..7."""
    import oracle
    q = np.arange(8, dtype=np.int8)[:, None]
    word = int(oracle.pack_int4(q - 0)[0, 0]) ^ 0x88888888   # nibble = code + 8
    got = 0
    for c in range(8):
        at, shift = kv.key_place(128, 0, 32 + 8 + c)         # j = 1, kb = 1: word 5
        assert at // 4 == 5
        got |= c << (8 * (at % 4) + shift)
    assert got == word


def test_quantiser_by_hand():
    x = np.array([0.0, 15.0, 7.4, 7.5, 8.5, 0.49, 14.6, 1.0] * 4, np.float32)   # lo 0, step 1
    q, step, lo = kv.quantise(x, 32)
    assert step[0] == 1 and lo[0] == 0
    assert list(q[:8]) == [0, 15, 7, 8, 8, 0, 15, 1]          # half to even
    q, step, lo = kv.quantise(np.full(32, -3.25, np.float32), 32)
    assert step[0] == 0 and lo[0] == np.float16(-3.25) and not q.any()
    assert (kv.dequantise(q, step, lo) == -3.25).all()


def test_quantiser_error_is_half_a_step():
    """|x' - x| <= step/2, plus the rounding of lo and step to fp16 at the clamped ends."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((500, 128)) * np.exp(rng.standard_normal((500, 1)))).astype(np.float32)
    q, step, lo = kv.quantise(x, 32)
    err = np.abs(kv.dequantise(q, step, lo).astype(np.float64) - x)
    s, low = (np.repeat(a.astype(np.float64), 32, -1) for a in (step, np.abs(lo)))
    # clamp: lo lies up to 2^-11 |lo| above min x; lo + 15 step up to 15 * 2^-11 step (or a subnormal's
    # half step) below max x; the quotient's own float32 roundings are far below
    assert (err <= s / 2 * (1 + 1e-5) + 2.0 ** -11 * low + 15 * (2.0 ** -11 * s + 2.0 ** -25)).all()


def test_step_on_a_tie_of_fp16():
    """The range times float32's 1/15, which lies above 1/15: 12.48828125, a tie, goes up to the odd neighbour."""
    x = np.linspace(-181.5, 15 * 12.48828125 - 181.5, 32, dtype=np.float32)
    _, step, _ = kv.quantise(x, 32)
    assert step[0] == 12.4921875


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 40000.0])
def test_rows_that_do_not_fit_read_back_as_nan(bad):
    c = kv.Cache(1, 2, 64, 32, 16)
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 2, 64)).astype(np.float32)
    v[1, 5] = bad
    c.write(0, 3, k, v)
    a, b = c.read(0, 3)
    assert np.isfinite(a[0]).all() and np.isfinite(b[0]).all()
    assert np.isnan(a[1]).all() and np.isnan(b[1]).all()


def test_largest_values_stay_inside_fp16():
    """lo + 15*step of any two ends within +-32768 rounds to at most 65504 in fp16."""
    rng = np.random.default_rng(2)
    ends = np.sort(rng.uniform(-32768, 32768, (20000, 2)), -1)
    ends[:4] = [[-32768, 32768], [32752, 32768], [-32768, -32752], [0, 32768]]
    x = np.repeat(ends, 16, -1).astype(np.float32)
    q, step, lo = kv.quantise(x, 32)
    top = kv.dequantise(np.full_like(q, 15), step, lo)
    assert np.isfinite(top.astype(np.float16)).all()


def test_attention_by_hand():
    c = kv.Cache(2, 1, 64, 64, 16)
    rows = np.zeros((2, 1, 64), np.float32)
    rows[0, 0, :2], rows[1, 0, :2] = (0, 15), (15, 0)
    for t in range(2):
        c.write(1, t, rows[t], rows[1 - t])
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = np.log(3.0) / 15
    table = np.array([[1]])
    o, lse, _, _ = kv.attention(c, q, None, [2], table, scale=1.0)
    assert np.allclose(o[0, 0, :2], [15, 0]) and np.isclose(lse[0, 0], 0)     # sees token 0 alone
    assert np.allclose(o[1, 0, :2], [15 / 4, 45 / 4]) and np.isclose(lse[1, 0], np.log(4))
    o, lse, _, _ = kv.attention(c, q, None, [1], table, scale=1.0)             # first row: no position
    assert not o[0].any() and lse[0, 0] == -np.inf and np.allclose(o[1, 0, 0], 15)


# ---- the library ------------------------------------------------------------

@pytest.fixture(scope="module")
def awq():
    from weight_only_quantization_awq_amd import awq
    awq._lib = None   # (load anew: a test that reloads the module puts back a library that knows the classes of before)
    return awq


def _cache(awq, **over):
    f = dict(pages=FAKE, n_pages=8, page_stride=4 * 16 * (128 + 8), heads=4, dim=128, group=128, page=16)
    f.update(over)
    return awq._KvCacheC(**f)


def _batch(awq, **over):
    f = dict(rows=6, batch=3, max_pages=4, row_start=None, kv_len=FAKE, block_table=FAKE)
    f.update(over)
    return awq._KvBatchC(**f)


def test_struct_layouts_match_the_header(tmp_path):
    from weight_only_quantization_awq_amd import awq
    src = tmp_path / "sizes.c"
    names = {"awq_kv_cache": awq._KvCacheC, "awq_kv_batch": awq._KvBatchC}
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


@built
@pytest.mark.parametrize("page,heads,dim,group", [(16, 8, 128, 128), (256, 1, 64, 32), (64, 5, 256, 64)])
def test_page_size(awq, page, heads, dim, group):
    assert awq.kv_page_size(page, heads, dim, group) == heads * kv.block_bytes(page, dim, group)


@built
@pytest.mark.parametrize("args", [(15, 8, 128, 128), (24, 8, 128, 128), (512, 8, 128, 128), (0, 8, 128, 128),
                                  (16, 0, 128, 128), (16, 65536, 128, 128), (16, 8, 96, 32), (16, 8, 0, 32),
                                  (16, 8, 64, 128), (16, 8, 128, 16), (16, 8, 128, 0), (16, 8, 256, 256)])
def test_page_size_refuses(awq, args):
    assert awq.load().awq_kv_page_size(*args) == 0
    assert awq.load().awq_last_error() != b""
    with pytest.raises(awq.AwqError):
        awq.kv_page_size(*args)


BAD_CACHE = [(dict(pages=None), ARG), (dict(pages=FAKE + 8), ARG), (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 31), SHAPE),
             (dict(page_stride=4 * 16 * 136 - 16), SHAPE), (dict(page_stride=4 * 16 * 136 + 8), SHAPE),
             (dict(heads=0), SHAPE), (dict(dim=96), SHAPE), (dict(group=48), ARG), (dict(page=20), ARG)]
BAD_BATCH = [(dict(batch=0), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=7), SHAPE), (dict(max_pages=0), SHAPE),
             (dict(max_pages=1 << 40), SHAPE), (dict(max_pages=(1 << 62)), SHAPE), (dict(batch=1 << 62, rows=0), SHAPE),
             (dict(rows=(1 << 62), row_start=FAKE), SHAPE), (dict(rows=1 << 26, row_start=FAKE), SHAPE),
             (dict(batch=1 << 20, rows=0), SHAPE), (dict(batch=1 << 20, rows=0, max_pages=1 << 16), SHAPE),
             (dict(kv_len=None), ARG), (dict(block_table=None), ARG), (dict(kv_len=FAKE + 2), ARG),
             (dict(block_table=FAKE + 1), ARG), (dict(row_start=FAKE + 2), ARG)]
EVERY = [("cache", o, s) for o, s in BAD_CACHE] + [("batch", o, s) for o, s in BAD_BATCH]


@built
@pytest.mark.parametrize("which,over,status", EVERY)
def test_refuses_bad_caches_and_batches(awq, which, over, status):
    lib = awq.load()
    c, b = _cache(awq, **(over if which == "cache" else {})), _batch(awq, **(over if which == "batch" else {}))
    for st in (lib.awq_kv_append(c, b, FAKE, FAKE, 1, 512, 512, None), lib.awq_kv_read(c, b, FAKE, FAKE, 1, 512, 512, None),
               lib.awq_kv_attention(c, b, FAKE, 1, 8, 1024, 2, 1.0, 1, 0, FAKE, 1024, None, FAKE, 1 << 40, None)):
        assert st == status
        assert lib.awq_last_error() != b""


@built
def test_refuses_null_structs(awq):
    lib = awq.load()
    for c, b in ((None, _batch(awq)), (_cache(awq), None)):
        assert lib.awq_kv_append(c, b, FAKE, FAKE, 1, 512, 512, None) == ARG
        assert lib.awq_kv_read(c, b, FAKE, FAKE, 1, 512, 512, None) == ARG
        assert lib.awq_kv_attention(c, b, FAKE, 1, 8, 1024, 2, 1.0, 1, 0, FAKE, 1024, None, None, 0, None) == ARG
        assert lib.awq_kv_attention_workspace_size(c, b, 8, 0) == 0 and lib.awq_last_error() != b""


@built
@pytest.mark.parametrize("K,V,t,ks,vs,status", [
    (None, FAKE, 1, 512, 512, ARG), (FAKE, None, 1, 512, 512, ARG), (FAKE + 8, FAKE, 1, 512, 512, ARG),
    (FAKE, FAKE + 2, 1, 512, 512, ARG), (FAKE, FAKE, 3, 512, 512, DTYPE), (FAKE, FAKE, -1, 512, 512, DTYPE),
    (FAKE, FAKE, 1, 511, 512, SHAPE), (FAKE, FAKE, 1, 512, 516, SHAPE), (FAKE, FAKE, 0, 512, 514, SHAPE),
    (FAKE, FAKE, 1, 1 << 40, 512, SHAPE), (FAKE, FAKE, 1, 512, -512, SHAPE)])
def test_copies_refuse(awq, K, V, t, ks, vs, status):
    lib = awq.load()
    assert lib.awq_kv_append(_cache(awq), _batch(awq), K, V, t, ks, vs, None) == status
    assert lib.awq_kv_read(_cache(awq), _batch(awq), K, V, t, ks, vs, None) == status


GOOD = dict(Q=FAKE, t=1, q_heads=8, q_stride=1024, max_rows=2, scale=0.5, causal=1, window=0, O=FAKE, o_stride=1024,
            lse=None, workspace=FAKE, size=1 << 40)


@built
@pytest.mark.parametrize("over,status", [
    (dict(Q=None), ARG), (dict(O=None), ARG), (dict(Q=FAKE + 4), ARG), (dict(O=FAKE + 8), ARG), (dict(lse=FAKE + 2), ARG),
    (dict(t=0), DTYPE), (dict(t=3), DTYPE), (dict(q_heads=0), SHAPE), (dict(q_heads=6), SHAPE), (dict(q_heads=65536), SHAPE),
    (dict(q_stride=1016), SHAPE), (dict(o_stride=1028), SHAPE), (dict(max_rows=-1), SHAPE), (dict(scale=0.0), ARG),
    (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(causal=2), ARG),
    (dict(window=-1), ARG), (dict(window=5, causal=0), ARG), (dict(workspace=None), WORKSPACE),
    (dict(workspace=FAKE + 8), WORKSPACE), (dict(size=100), WORKSPACE)])
def test_attention_refuses(awq, over, status):
    lib = awq.load()
    a = dict(GOOD, **over)
    b = _batch(awq, max_pages=64)   # long enough for a workspace
    st = lib.awq_kv_attention(_cache(awq), b, a["Q"], a["t"], a["q_heads"], a["q_stride"], a["max_rows"], a["scale"],
                              a["causal"], a["window"], a["O"], a["o_stride"], a["lse"], a["workspace"], a["size"], None)
    assert st == status
    assert lib.awq_last_error() != b""


@built
def test_no_rows_is_a_call_without_launches(awq):
    lib = awq.load()
    b = _batch(awq, rows=0)
    assert lib.awq_kv_append(_cache(awq), b, None, None, 1, 512, 512, None) == 0
    assert lib.awq_kv_read(_cache(awq), b, None, None, 1, 512, 512, None) == 0
    assert lib.awq_kv_attention(_cache(awq), b, None, 1, 8, 1024, 0, 1.0, 1, 0, None, 1024, None, None, 0, None) == 0
    assert lib.awq_last_error() == b""


@built
def test_short_tables_need_no_workspace(awq):
    lib = awq.load()
    # 12 pages of 16 tokens: 6 tiles of 32, never cut; a longer one can be
    assert lib.awq_kv_attention_workspace_size(_cache(awq), _batch(awq, max_pages=12), 8, 0) == 0
    assert lib.awq_last_error() == b""
    assert lib.awq_kv_attention_workspace_size(_cache(awq), _batch(awq, max_pages=13), 8, 0) > 0
    assert lib.awq_kv_attention_workspace_size(_cache(awq), _batch(awq, max_pages=13), 6, 0) == 0
    assert b"q_heads" in lib.awq_last_error()


@built
def test_workspace_is_bounded_whatever_the_length(awq):
    """The split path's pieces depend on the workers, not on the sequences' lengths."""
    lib = awq.load()
    size = [lib.awq_kv_attention_workspace_size(_cache(awq), _batch(awq, rows=8, batch=8, max_pages=n), 32, 0)
            for n in (1 << 10, 1 << 13, 1 << 16)]
    assert size[0] == size[1] == size[2] < 64 << 20


@built
def test_python_refusals(awq):
    import torch
    with pytest.raises(TypeError):
        awq.KvCache(torch.zeros(4, 8, 2176), 128)
    with pytest.raises(ValueError):
        awq.KvCache(torch.zeros(4, 8, 2177, dtype=torch.uint8), 128)
    with pytest.raises(ValueError):
        awq.KvCache(torch.zeros(4, 2176, 8, dtype=torch.uint8).transpose(1, 2), 128)
    with pytest.raises(awq.AwqError):
        awq.KvCache(torch.zeros(4, 8, 2176, dtype=torch.uint8), 100)
    c = awq.KvCache(torch.zeros(4, 8, 2176, dtype=torch.uint8), 128)     # a CPU pool cannot be used
    assert c.heads == 8
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        awq.kv_append(c, torch.zeros(1, 8, 128), torch.zeros(1, 8, 128), i.view(1, 1), i)
    with pytest.raises(ValueError):
        awq.kv_attention(torch.zeros(1, 8, 128, dtype=torch.bfloat16), c, i.view(1, 1), i)
