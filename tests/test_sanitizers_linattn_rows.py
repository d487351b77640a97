"""Launch plans of linear attention for packed rows under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only), with stub launchers."""

import os
import subprocess

import pytest

from tests.test_sanitizers_linattn import ROOT, SAN


@pytest.mark.skipif(not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"), reason="no HIP headers")
def test_packed_rows_are_laid_out_for_their_tokens(tmp_path):
    csrc = os.path.join(ROOT, "rwkv_wkv7_delta_amd", "csrc")
    exe = str(tmp_path / "linattn_rows_driver")
    build = subprocess.run(
        ["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include",
         "-D__HIP_PLATFORM_AMD__", "-o", exe, os.path.join(ROOT, "tests", "sanitize", "linattn_rows_driver.cpp"),
         os.path.join(csrc, "wkv7_linattn_api.cpp")], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0 and " 0 failed checks" in run.stdout, run.stdout[-2000:] + run.stderr[-4000:]
