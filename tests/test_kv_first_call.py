"""kv_tables takes no cache, so it may be the first call of a program: it loads the library itself (CPU)."""
from __future__ import annotations

import pytest
import torch

from tests.test_kv_step_cpu import built


class Ints:
    """What the binding asks of an int32 tensor on a GPU."""
    device, dtype = torch.device("cuda", 0), torch.int32

    def __init__(self, *shape):
        self.shape = torch.Size(shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def dim(self):
        return len(self.shape)


@built
def test_kv_tables_loads_the_library(monkeypatch):
    from weight_only_quantization_awq_amd import awq
    calls = []
    monkeypatch.setattr(awq, "_lib", None)
    monkeypatch.setattr(awq, "_kv_call", lambda device, fn, *args: calls.append((device, fn, len(args))))
    out = awq.KvStep(Ints(2), Ints(3), Ints(1), None, None)
    assert awq.kv_tables(Ints(2, 4), Ints(2), Ints(2), Ints(5), page=16, out=out) is out
    (device, fn, count), = calls
    assert device == Ints.device and fn is awq.load().awq_kv_tables_ex and count + 1 == len(fn.argtypes)


@pytest.mark.gpu
def test_kv_tables_as_a_program_s_first_call(monkeypatch):
    from weight_only_quantization_awq_amd import awq
    monkeypatch.setattr(awq, "_lib", None)
    x = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    assert awq.kv_tables(x, x[0], x[0] + 1, x[0] + 7).kv_len.tolist() == [1] and x.tolist() == [[7]]
