"""Rules of the 4-bit key/value cache, pinned on the oracle (CPU, no GPU)."""
from __future__ import annotations

import numpy as np

from oracle import kv_oracle as kv


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
