"""Rows that share memory (CPU): kv_rows_meet against a map of every byte, under sanitizers."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from tests.test_sanitizers import BASE, CSRC, HIPCC, ROOT, SAN


@pytest.mark.timeout(300)
def test_rows_that_share_memory_are_found(tmp_path):
    if not os.path.exists(HIPCC) or shutil.which("c++filt") is None:
        pytest.skip("ROCm toolchain not present")
    exe = str(tmp_path / "kv_meet_driver")
    r = subprocess.run([HIPCC, *BASE, *SAN, "-I", CSRC, os.path.join(ROOT, "tests", "sanitizer", "kv_meet_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-2000:])
