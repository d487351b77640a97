"""The distances of tests/test_lane_hazards.py along every path through a compiled scan
kernel (hipcc, no GPU needed): over loops' back edges and from each branch to its target,
where a walk along the listing sees only the instruction written above."""

import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

from rwkv_wkv7_delta_amd import build as hip_build
from tests.test_lane_hazards import SOURCES, SWAP, TRANS, _operands, _regs

OTHER = (frozenset(), False)   # an instruction that writes no vector register
LEAVES = re.compile(r"s_(branch|endpgm|setpc)")


def kernels(asm):
    """(name, blocks, successors of each) of every function in a listing."""
    name, items = None, []
    for raw in asm.splitlines():
        line = raw.split(";")[0].strip()
        if (m := re.match(r"(_Z\w+):", line)):
            name, items = m.group(1), []
        elif name and line.startswith(".Lfunc_end"):
            yield name, *blocks_of(items)
            name = None
        elif name and line and (line.startswith(".LBB") or line[0] not in "._"):
            items.append(line)


def blocks_of(items):
    blocks, label = [[]], {}
    for line in items:
        if line.endswith(":"):
            if blocks[-1]:
                blocks.append([])
            label[line[:-1]] = len(blocks) - 1
        else:
            blocks[-1].append(line)
            if re.match(r"s_(cbranch|branch|endpgm|setpc)", line):
                blocks.append([])
    follow = []
    for k, block in enumerate(blocks):
        last = block[-1] if block else ""
        to = [label[m.group(1)]] if (m := re.match(r"s_(?:cbranch_\w+|branch)\s+(\S+)", last)) else []
        if not LEAVES.match(last) and k + 1 < len(blocks):
            to.append(k + 1)
        follow.append(to)
    return blocks, follow


def after(seen, line, bad):
    """The two instructions behind `line`, from those before it; what comes too soon goes to bad."""
    if line.startswith("s_nop"):
        return (seen + (OTHER,) * (int(line.split()[1], 0) + 1))[-2:]
    if not line.startswith("v_") or len(line.split(None, 1)) < 2:
        return (seen + (OTHER,))[-2:]
    writes, reads = _operands(line)
    near = set().union(*(w for w, _ in seen))
    if "_dpp" in line:
        source = re.split(r" row_| quad_perm", line.split(None, 1)[1])[0].split(",")[1]
        if _regs(source) & near:
            bad.add(("DPP", line))
    if SWAP.match(line) and reads & near:
        bad.add(("swap", line))
    if seen and seen[-1][1] and not TRANS.match(line) and reads & seen[-1][0]:
        bad.add(("transcendental", line))
    return (seen + ((frozenset(writes), bool(TRANS.match(line))),))[-2:]


def hazards(blocks, follow):
    """Every block from every pair of instructions that some path leaves in front of it."""
    entry = [set() for _ in blocks]
    entry[0].add(())
    todo, bad = [(0, ())], set()
    while todo:
        k, seen = todo.pop()
        for line in blocks[k]:
            seen = after(seen, line, bad)
        for n in follow[k]:
            if seen not in entry[n]:
                entry[n].add(seen)
                todo.append((n, seen))
    return bad


def test_paths_through_a_loop():
    loop = ["s_mov_b32 s0, 0", ".LBB0_1:", "v_add_f32_dpp v3, v1, v1 row_ror:8 row_mask:0xf bank_mask:0xf",
            "v_mov_b32_e32 v4, v5", "v_mov_b32_e32 {w}, v2", "s_cbranch_scc1 .LBB0_1", "s_endpgm"]
    for written, want in (("v1", {"DPP"}), ("v6", set())):
        got = hazards(*blocks_of([line.format(w=written) for line in loop]))
        assert {rule for rule, _ in got} == want
    skip = ["v_exp_f32_e32 v1, v2", "s_cbranch_scc1 .LBB0_2", "s_nop 3", ".LBB0_2:", "v_mul_f32_e32 v3, v1, v1",
            "s_endpgm"]
    assert hazards(*blocks_of(skip)) == set()   # the branch itself lies between
    swap = ["v_mov_b32_e32 v1, v2", "s_cbranch_scc1 .LBB0_2", "s_nop 3", ".LBB0_2:", "v_permlane32_swap_b32_e32 v4, v1",
            "s_endpgm"]
    assert {rule for rule, _ in hazards(*blocks_of(swap))} == {"swap"}


@pytest.mark.skipif(not os.path.exists(hip_build.HIPCC) and not shutil.which("hipcc"), reason="no hipcc")
def test_distances_hold_on_every_path(tmp_path):
    def listing(src):
        out = str(tmp_path / (src + ".s"))
        res = subprocess.run([hip_build.HIPCC, *hip_build.COMMON, "-x", "hip", "-S", "--offload-device-only",
                              os.path.join(hip_build.CSRC, src), "-o", out], capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        with open(out) as f:
            return f.read()

    with concurrent.futures.ThreadPoolExecutor() as pool:
        for src, asm in zip(SOURCES, pool.map(listing, SOURCES)):
            found = 0
            for name, blocks, follow in kernels(asm):
                found += 1
                assert sum(map(len, follow)) > 0 and blocks[0], name
                bad = hazards(blocks, follow)
                assert not bad, f"{name}: {len(bad)}: {sorted(bad)[:5]}"
            assert found > 20, (src, found)
