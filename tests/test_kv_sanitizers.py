"""Host-side sanitizers over the key/value cache's validation and sizing (CPU,
no GPU): awq_kv.hip under AddressSanitizer and UndefinedBehaviorSanitizer on the
host side, driven by tests/sanitizer/kv_driver.cpp."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from tests.test_sanitizers import BASE, CSRC, HIPCC, KERNELS, ROOT, SAN, _kernel_object

KV_KERNELS = ["k_kv", "k_kv_attend_64", "k_kv_attend_128", "k_kv_attend_256"]


@pytest.mark.timeout(600)
def test_kv_validation_under_host_sanitizers(tmp_path):
    if not os.path.exists(HIPCC) or shutil.which("c++filt") is None:
        pytest.skip("ROCm toolchain not present")
    tmp = str(tmp_path)
    objs = []
    for src in (os.path.join(CSRC, "awq_api.hip"), os.path.join(CSRC, "awq_kv.hip"),
                os.path.join(ROOT, "tests", "sanitizer", "kv_driver.cpp")):
        objs.append(os.path.join(tmp, os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, *BASE, *SAN, "-c", src, "-o", objs[-1]], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    objs += [_kernel_object(k, tmp) for k in KERNELS + KV_KERNELS]
    exe = os.path.join(tmp, "kv_driver")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "sanitized key/value cache checks passed" in r.stdout
