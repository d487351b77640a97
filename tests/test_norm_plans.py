"""The sizes of the group norm's tests of many rows make its workgroups go over their rows several
times (CPU only: the launch plans, with stub launchers, under sanitizers)."""

import os
import subprocess

import pytest

import rwkv_wkv7_delta_amd as wk
from tests.test_gpu_gnorm_modes import BACKWARD, FORWARD
from tests.test_sanitizers_linattn import ROOT, SAN


@pytest.mark.skipif(not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"), reason="no HIP headers")
def test_many_rows_are_several_passes(tmp_path):
    csrc = os.path.join(ROOT, "rwkv_wkv7_delta_amd", "csrc")
    exe = str(tmp_path / "norm_plans")
    build = subprocess.run(
        ["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include",
         "-D__HIP_PLATFORM_AMD__", "-o", exe, os.path.join(ROOT, "tests", "sanitize", "norm_plans_driver.cpp"),
         os.path.join(csrc, "wkv7_gnorm_api.cpp")], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    cases = [(*size, dtype, back) for sizes, back in ((BACKWARD, 1), (FORWARD, 0)) for size in sizes
             for dtype in (wk.WKV7_F32, wk.WKV7_BF16)]
    run = subprocess.run([exe, *[str(x) for c in cases for x in c]], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stderr[-4000:]
    plans = [tuple(map(int, line.split())) for line in run.stdout.splitlines()]
    assert len(plans) == len(cases)
    for c, (passes, ragged) in zip(cases, plans):
        assert passes >= 3 and ragged, (c, passes, ragged)
