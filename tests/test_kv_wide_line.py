"""Units, lines, pieces and joins of attention on the wide path (CPU, no GPU): awq_kv.hip's host code under sanitizers,
and the kernels' own arithmetic walked on the host by tests/sanitizer/kv_wide_driver.cpp."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from tests.test_sanitizers import BASE, CSRC, HIPCC, KERNELS, ROOT, SAN, _kernel_object


@pytest.mark.timeout(600)
def test_every_unit_is_made_up_of_its_pieces(tmp_path):
    if not os.path.exists(HIPCC) or shutil.which("c++filt") is None:
        pytest.skip("ROCm toolchain not present")
    tmp = str(tmp_path)
    objs = []
    for src in [os.path.join(CSRC, x) for x in ("awq_api.hip", "awq_kv.hip")] + [
            os.path.join(ROOT, "tests", "sanitizer", "kv_wide_driver.cpp")]:
        objs.append(os.path.join(tmp, os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, *BASE, *SAN, "-I", CSRC, "-c", src, "-o", objs[-1]], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    objs += [_kernel_object(k, tmp) for k in KERNELS]
    exe = os.path.join(tmp, "kv_wide_driver")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=400)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "columns joined" in r.stdout
