"""The pool's size as a step's tables take it, without a GPU."""
from __future__ import annotations

import pytest

from tests.test_kv_step_cpu import ARG, SHAPE, awq, built  # noqa: F401  (awq: a fixture)


def _tables(awq, n_pages, kv_len=0x1000):
    step = awq._KvStepC(0x6000, 0x7000, 0x8000, 0x9000, 0xA000)
    return awq.load().awq_kv_tables_ex(16, 3, 4, kv_len, 0x2000, 0x3000, 5, 0x4000, 0x5000, 7, n_pages, step, None)


@built
@pytest.mark.parametrize("n_pages", [-1, 1 << 31, -(1 << 63), (1 << 63) - 1])
def test_tables_refuse_sizes_of_a_pool(awq, n_pages):
    assert _tables(awq, n_pages) == SHAPE
    assert b"n_pages" in awq.load().awq_last_error()


@built
@pytest.mark.parametrize("kv_len", [None, 0x1002, 0x6000])
def test_tables_with_a_size_refuse_what_they_do_without(awq, kv_len):
    assert _tables(awq, 40, kv_len) == ARG
