"""What reads a matrix instruction's result waits for it, along every path (no
GPU needed): the listing of the routed layer's kernels, built here from source.

The compiler puts wait states behind a matrix instruction, but not where a
branch is taken between it and the reader: a sum that had been moved behind such
a branch was taken of registers that were not written yet.  The source keeps
every sum in front of the next branch; this test looks at what came of it.
Behind the instructions used here (16 x 16, 4 or 8 passes) the compiler itself
leaves 8 states or more."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "conv_implicit_gemm_amd", "csrc")
STATES = 8


def vgprs(word):
    m = re.match(r"v\[(\d+):(\d+)\]$|v(\d+)$", word)
    if not m:
        return set()
    return {int(m.group(3))} if m.group(3) else set(range(int(m.group(1)), int(m.group(2)) + 1))


def functions(listing):
    """name -> (instructions as word lists, label -> index)"""
    name, found = None, {}
    for line in listing.split("\n"):
        line = line.split(";")[0].strip()
        m = re.match(r"(_Z\w+):$", line)
        if m:
            name = m.group(1)
            found[name] = ([], {})
        elif name is None or not line:
            continue
        elif re.match(r"\.LBB\w+:$", line):
            found[name][1][line[:-1]] = len(found[name][0])
        elif not line.startswith(".") and not line.endswith(":"):
            found[name][0].append(re.split(r"[ ,]+", line))
    return found


def early_reads(code, labels):
    """(matrix instruction, reader, states between) of every read that comes too early"""
    for start, first in enumerate(code):
        if not first[0].startswith("v_mfma"):
            continue
        result, seen, todo = vgprs(first[1]), {}, [(start + 1, 0)]
        while todo:
            at, states = todo.pop()
            if at >= len(code) or states >= STATES or seen.get(at, STATES) <= states:
                continue
            seen[at] = states
            op, args = code[at][0], code[at][1:]
            if op == "s_endpgm":
                continue
            if op.startswith("v_mfma"):
                if (vgprs(args[1]) | vgprs(args[2])) & result:
                    yield first, code[at], states
                    continue
                if vgprs(args[0]) & result:      # the next of its chain, or a new one
                    continue
            elif op.startswith(("v_", "global_", "flat_", "buffer_", "scratch_", "ds_")):
                store = "store" in op or "write" in op
                if set().union(*map(vgprs, args if store else args[1:])) & result:
                    yield first, code[at], states
                    continue
                if args and not store and vgprs(args[0]) & result:
                    continue
            if op.startswith(("s_branch", "s_cbranch")):
                todo.append((labels[args[0]], states + 1))
            if op != "s_branch":
                todo.append((at + 1, states + (int(args[0], 0) + 1 if op == "s_nop" else 1)))


def test_the_reader_finds_reads_behind_a_taken_branch():
    code = """
_Zkernel:
	v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0
	s_cbranch_scc1 .LBB0_1
	s_nop 7
	v_add_f32_e32 v4, v0, v4
.LBB0_1:
	v_add_f32_e32 v5, v1, v5
	s_endpgm
"""
    found = list(early_reads(*functions(code)["_Zkernel"]))
    assert [(r[1], s) for _, r, s in found] == [("v5", 1)]


def test_sums_wait_for_the_matrix_unit(tmp_path):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not shutil.which(hipcc):
        pytest.skip("needs hipcc")
    out = str(tmp_path / "k_moe.s")
    subprocess.run([hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", "-I" + CSRC, "--cuda-device-only", "-S", os.path.join(CSRC, "k_moe.hip"), "-o", out],
                   check=True, stderr=subprocess.DEVNULL)
    with open(out) as f:
        kernels = functions(f.read())
    assert sum("moe_" in name for name in kernels) >= 14
    for name, (code, labels) in kernels.items():
        early = list(early_reads(code, labels))
        assert not early, "%s: %s" % (name, early[:3])
