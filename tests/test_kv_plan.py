"""The attention's pieces in its workspace (CPU, no GPU): awq_kv.hip's plan and the
split path's own arithmetic, walked on the host under sanitizers by
tests/sanitizer/kv_plan_driver.cpp, sequences with more rows than max_rows among them."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from tests.test_sanitizers import BASE, CSRC, HIPCC, KERNELS, ROOT, SAN, _kernel_object


@pytest.mark.timeout(600)
def test_every_piece_has_its_own_place(tmp_path):
    if not os.path.exists(HIPCC) or shutil.which("c++filt") is None:
        pytest.skip("ROCm toolchain not present")
    tmp = str(tmp_path)
    objs = []
    for src in (os.path.join(CSRC, "awq_api.hip"), os.path.join(CSRC, "awq_kv.hip"),
                os.path.join(ROOT, "tests", "sanitizer", "kv_plan_driver.cpp")):
        objs.append(os.path.join(tmp, os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, *BASE, *SAN, "-I", CSRC, "-c", src, "-o", objs[-1]], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    objs += [_kernel_object(k, tmp) for k in KERNELS]
    exe = os.path.join(tmp, "kv_plan_driver")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "pieces in their places" in r.stdout


@pytest.mark.timeout(600)
def test_schedule_of_the_wide_path(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("ROCm toolchain not present")
    exe = str(tmp_path / "kv_schedule_driver")
    r = subprocess.run([HIPCC, *BASE, "-I", CSRC, os.path.join(ROOT, "tests", "sanitizer", "kv_schedule_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "schedules hold" in r.stdout, r.stdout
