"""Static checks of the scan kernels' lane operations (hipcc, no GPU needed).

The scan's kernels hold vector instructions with DPP operands and lane swaps next
to each other in inline assembly, where the compiler keeps no distance between
them.  In every compiled kernel, walked linearly:

1. the register that an instruction reads through DPP was written by neither of
   the two instructions before it;
2. nor were the two that a lane swap exchanges;
3. the instruction right behind a transcendental one does not read its result
   (another transcendental may).

Instructions of every kind count, an s_nop n as n + 1.
"""

import os
import re
import shutil
import subprocess

import pytest

from rwkv_wkv7_delta_amd import build as hip_build

SOURCES = ["wkv7_ssm.hip", "wkv7_ssm_bwd.hip"]
TRANS = re.compile(r"v_(exp|log|rcp|rsq|sqrt|sin|cos)_f32")
SWAP = re.compile(r"v_permlane\d+_swap")


def _regs(text):
    out = set()
    for one, lo, hi in re.findall(r"\bv(?:(\d+)|\[(\d+):(\d+)\])", text):
        out.update([int(one)] if one else range(int(lo), int(hi) + 1))
    return out


def _operands(line):
    """(registers written, registers read) of a vector instruction."""
    name, rest = line.split(None, 1)
    ops = [o.strip() for o in rest.split(",")]
    if SWAP.match(name):
        both = _regs(rest)
        return both, both
    return _regs(ops[0]), _regs(",".join(ops[1:]))


def hazards(asm):
    """(rule, line) of every instruction that comes too soon."""
    bad, seen = [], []   # seen: (registers written, transcendental) of the instructions before
    for raw in asm.splitlines():
        line = raw.strip()
        if line.startswith("s_nop"):
            seen += [(set(), False)] * (int(line.split()[1], 0) + 1)
            continue
        if not line or line[0] in ".;_" or line.endswith(":"):
            continue
        if not line.startswith("v_") or len(line.split(None, 1)) < 2:
            seen.append((set(), False))
            continue
        writes, reads = _operands(line)
        near = set().union(*(w for w, _ in seen[-2:]))
        if "_dpp" in line:
            source = re.split(r" row_| quad_perm", line.split(None, 1)[1])[0].split(",")[1]
            if _regs(source) & near:
                bad.append(("DPP", line))
        if SWAP.match(line) and reads & near:
            bad.append(("swap", line))
        if seen and seen[-1][1] and not TRANS.match(line) and reads & seen[-1][0]:
            bad.append(("transcendental", line))
        seen = seen[-2:] + [(writes, bool(TRANS.match(line)))]
    return bad


def test_what_counts_as_too_soon():
    far = "v_mov_b32_e32 v1, v2\ns_nop 1\n"
    near = "v_mov_b32_e32 v1, v2\ns_nop 0\n"
    dpp = "v_add_f32_dpp v3, v1, v1 row_ror:8 row_mask:0xf bank_mask:0xf\n"
    swap = "v_permlane32_swap_b32_e32 v4, v1\n"
    assert hazards(far + dpp + swap) == []
    assert [r for r, _ in hazards(near + dpp)] == ["DPP"]
    assert [r for r, _ in hazards(near + swap)] == ["swap"]
    assert [r for r, _ in hazards("v_exp_f32_e32 v1, v2\nv_mul_f32_e32 v3, v1, v1\n")] == ["transcendental"]
    assert hazards("v_exp_f32_e32 v1, v2\ns_nop 0\nv_mul_f32_e32 v3, v1, v1\n") == []


@pytest.mark.skipif(not os.path.exists(hip_build.HIPCC) and not shutil.which("hipcc"), reason="no hipcc")
@pytest.mark.parametrize("src", SOURCES)
def test_lane_operations_keep_their_distance(src, tmp_path):
    out = str(tmp_path / "k.s")
    res = subprocess.run([hip_build.HIPCC, *hip_build.COMMON, "-x", "hip", "-S", "--offload-device-only",
                          os.path.join(hip_build.CSRC, src), "-o", out], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    with open(out) as f:
        asm = f.read()
    assert "_dpp" in asm
    bad = hazards(asm)
    assert not bad, f"{len(bad)}: {bad[:5]}"
