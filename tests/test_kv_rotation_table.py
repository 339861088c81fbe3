"""The table of angles where its sizes are at their ends (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_kv_step_cpu import awq, built  # noqa: F401  (awq: a fixture)


@built
@pytest.mark.parametrize("rot", [15, 1, -1, -16])
def test_channels_come_in_pairs(awq, rot):
    """An odd number gave a table of one channel more, at the frequencies of neither."""
    with pytest.raises(ValueError, match="rot"):
        awq.kv_rotation_table(4, rot, device="cpu")


@built
@pytest.mark.parametrize("positions,rot", [(0, 16), (1, 16), (5, 0), (3, 256)])
def test_sizes(awq, positions, rot):
    t = awq.kv_rotation_table(positions, rot, device="cpu").numpy()
    assert t.shape == (positions, 2, rot // 2) and t.dtype == np.float32
    assert (t[:1, 0] == 1).all() and (t[:1, 1] == 0).all()
