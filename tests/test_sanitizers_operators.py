"""The C ABI of the operators around the layer, host code under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): operators_api.hip with stand-ins for the launches, driven
by tests/sanitize/operators_driver.cpp.  A sanitizer report ends the driver, so its exit status
and closing line are the whole check."""
import os
import subprocess

import pytest

from tests.test_sanitizers import CSRC, ENV, HIPCC, SAN


def test_operator_argument_paths_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "operators_driver")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-x", "hip",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer",
           "-o", exe, os.path.join(SAN, "operators_driver.cpp"), os.path.join(CSRC, "operators_api.hip")]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], env=ENV, timeout=120, capture_output=True, text=True)
    assert r.returncode == 0 and "checks passed" in r.stdout, r.stdout + r.stderr
