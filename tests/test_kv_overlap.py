"""Where the outputs of the rotated append and of attention may lie (CPU): what is refused before any HIP call."""
from __future__ import annotations

import pytest

from tests.test_kv_view_cpu import PREFIX, _call
from tests.test_kv_step_cpu import ARG, FAKE, _batch, _rotated, awq, built  # noqa: F401  (awq: a fixture)

HEAD, ROW = 128 * 2, 1024 * 2   # bytes of a head and of a row of 8, bf16


@built
@pytest.mark.parametrize("out,out_stride", [
    (FAKE + HEAD, 1024),                  # a head further on
    (FAKE - HEAD, 1024),                  # a head before
    (FAKE + ROW, 1024),                   # the next row
    (FAKE + 5 * ROW + ROW // 2, 1024),    # half of the last row
    (FAKE - 5 * ROW - 16, 1024),          # all but 16 bytes of its last row before, 16 in the first
    (FAKE + 16, 1024),
    (FAKE + ROW, 2048),                   # another stride, rows that come to lie on later ones
])
def test_an_output_over_other_queries_is_refused(awq, out, out_stride):
    """6 rows of 8 heads of 128, bf16, contiguous."""
    assert _rotated(awq, out=out, out_stride=out_stride) == ARG
    assert b"share memory" in awq.load().awq_last_error()


@built
def test_a_fused_projection_a_head_further_on_is_refused(awq):
    """Rows of 8 query heads and 2 * 4 others: the output begins one head behind the queries, and 9 of 8 would fit."""
    assert _rotated(awq, q_stride=2048, k_stride=2048, v_stride=2048, k=FAKE + 8 * HEAD, v=FAKE + 12 * HEAD, out=FAKE + HEAD,
                    out_stride=2048) == ARG
    assert b"share memory" in awq.load().awq_last_error()
    # and where the last row alone is met
    assert _rotated(awq, q_stride=2048, out=FAKE + 5 * 2 * ROW + 7 * HEAD, out_stride=2048) == ARG
    # no rows, nothing to share
    assert _rotated(awq, batch=_batch(awq, rows=0), out=FAKE + HEAD) == 0


@built
@pytest.mark.parametrize("view", [{}, dict(window=5, sinks=1), PREFIX], ids=["plain", "sinks", "prefix"])
@pytest.mark.parametrize("out,out_stride", [(FAKE + HEAD, 1024), (FAKE - HEAD, 1024), (FAKE + 5 * ROW, 1024), (FAKE, 2048), (FAKE + 16, 1024)])
def test_attention_over_other_queries_is_refused(awq, view, out, out_stride):
    assert _call(awq, out=out, out_stride=out_stride, **view) == ARG
    assert b"share memory" in awq.load().awq_last_error()
