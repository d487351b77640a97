"""The host code of the convolution and the scan (``wkv7_ssm_api.cpp``) under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): validation, segment
plans and size arithmetic over descriptors up to the integer limits, with stub
launchers that check grids, segments and 32-bit offsets of what would be launched."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]


@pytest.mark.skipif(not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"), reason="no HIP headers")
def test_mixers_abi_under_sanitizers(tmp_path):
    csrc = os.path.join(ROOT, "rwkv_wkv7_delta_amd", "csrc")
    exe = str(tmp_path / "mixers_driver")
    build = subprocess.run(
        ["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include",
         "-D__HIP_PLATFORM_AMD__", "-o", exe, os.path.join(ROOT, "tests", "sanitize", "mixers_driver.cpp"),
         os.path.join(csrc, "wkv7_ssm_api.cpp")], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0 and " 0 failed checks" in run.stdout, run.stdout[-2000:] + run.stderr[-4000:]
