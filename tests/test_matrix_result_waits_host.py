"""What reads a matrix instruction's result waits for it, along every path, in
all kernels of the experts' products and of the routed layer (no GPU needed):
listings built here from source.

As test_matrix_waits_host.py, which looks at one file for 8 states behind every
instruction and at plain operands, and stricter: the states go by the
instruction, operands count with their signs and magnitudes (-v0, |v0|), in
accumulation registers (a[0:3]) and where they are read beside being written
(v_fmac) or written by a vector instruction while the result is still to come."""
import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "conv_implicit_gemm_amd", "csrc")
UNITS = ["k_moe", "k_expert_i8", "k_expert_bf16", "k_expert_fp8", "k_expert_f32"]
# States between an instruction and a vector or memory instruction that reads its
# result: of the instructions with 4 passes, and with 8 (fp32's are two fewer).
STATES = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_i32_16x16x64_i8": 8, "v_mfma_f32_16x16x128_f8f6f4": 12,
          "v_mfma_f32_16x16x4_f32": 10}
MEMORY = ("global_", "flat_", "buffer_", "scratch_", "ds_")
BOTH = re.compile(r"v_(fmac|mac|pk_fmac|dot\w*c|swap)")      # what they write they read too


def registers(word):
    """The vector and accumulation registers that an operand names."""
    word = re.sub(r"^(-|neg\(|abs\(|sext\(|\|)+|[|)]+$", "", word)
    m = re.match(r"([va])(?:\[(\d+):(\d+)\]|(\d+))$", word)
    if not m:
        return frozenset()
    lo, hi = (m.group(4), m.group(4)) if m.group(4) else (m.group(2), m.group(3))
    return frozenset((m.group(1), n) for n in range(int(lo), int(hi) + 1))


def of(words):
    return frozenset().union(*map(registers, words))


class Code:
    """A function's instructions: names, registers read, written, operands, and labels."""

    def __init__(self):
        self.ops, self.args, self.labels = [], [], {}

    def add(self, words):
        self.ops.append(words[0])
        self.args.append(words[1:])


def functions(listing):
    code, found = None, {}
    for line in listing.split("\n"):
        line = line.split(";")[0].strip()
        m = re.match(r"(_Z\w+):$", line)
        if m:
            code = found[m.group(1)] = Code()
        elif code is None or not line:
            continue
        elif re.match(r"\.LBB\w+:$", line):
            code.labels[line[:-1]] = len(code.ops)
        elif not line.startswith(".") and not line.endswith(":"):
            code.add([w for w in re.split(r"[ ,\t]+", line) if w])
    return found


def touched_early(op, args, result):
    """Whether an instruction reads `result`, or (a vector one) writes it."""
    if op.startswith("v_mfma"):
        # the sums that it starts from may be the result itself, not a part of it
        sums = registers(args[3])
        return bool(of(args[1:3]) & result) or (sums != result and bool(sums & result))
    if op.startswith("v_"):
        return bool(of(args) & result)
    if op.startswith(MEMORY):
        all_read = "store" in op or "write" in op or "lds" in args or not op.startswith(("global_load", "flat_load", "buffer_load",
                                                                                      "scratch_load", "ds_"))
        return bool(of(args if all_read else args[1:]) & result)
    return False


def early(code):
    """(matrix instruction, the one that comes too early, states between)"""
    for start, first in enumerate(code.ops):
        if not first.startswith("v_mfma"):
            continue
        need, result = STATES[first], registers(code.args[start][0])
        assert len(result) == 4, (first, code.args[start])
        seen, todo = {}, [(start + 1, 0)]
        while todo:
            at, states = todo.pop()
            if at >= len(code.ops) or states >= need or seen.get(at, need) <= states:
                continue
            seen[at] = states
            op, args = code.ops[at], code.args[at]
            if op == "s_endpgm":
                continue
            if touched_early(op, args, result):
                yield (first, *code.args[start]), (op, *args), states
                continue
            if op.startswith("v_mfma") and registers(args[0]) & result:
                continue                    # the next of its chain, or a new one: looked at by itself
            if op.startswith(("s_branch", "s_cbranch")):
                todo.append((code.labels[args[0]], states + 1))
            assert not op.startswith(("s_setpc", "s_swappc", "s_call")), op
            if op != "s_branch":
                todo.append((at + 1, states + (int(args[0], 0) + 1 if op == "s_nop" else 1)))


def found_in(body):
    return [(r[0], s) for _, r, s in early(functions("_Zkernel:\n%s\n\ts_endpgm\n" % body)["_Zkernel"])]


BF16, F32 = "\tv_mfma_f32_16x16x32_bf16 %s, v[8:11], v[12:15], 0\n", "\tv_mfma_f32_16x16x4_f32 %s, v8, v12, 0\n"


@pytest.mark.parametrize("result,reader", [
    ("v[0:3]", "v_sub_f32_e64 v4, -v0, v5"), ("v[0:3]", "v_max_f32_e64 v4, |v0|, v5"), ("v[0:3]", "v_fma_f32 v4, v5, -|v3|, v6"),
    ("a[0:3]", "v_accvgpr_read_b32 v4, a0"), ("a[0:3]", "global_store_dwordx4 v4, a[0:3], s[0:1]"),
    ("v[0:3]", "v_fmac_f32_e32 v1, v5, v6"), ("v[0:3]", "v_mov_b32_e32 v1, 0"), ("v[0:3]", "ds_write_b128 v4, v[0:3]"),
    ("v[0:3]", "ds_bpermute_b32 v4, v5, v2"), ("v[0:3]", "buffer_load_dwordx4 v0, s[0:3], 0 offen lds"),
    ("v[0:3]", "global_atomic_add v4, v2, s[0:1]"), ("v[0:3]", "v_readfirstlane_b32 s0, v3"),
    ("v[0:3]", "v_mfma_f32_16x16x32_bf16 v[16:19], v[0:3], v[12:15], 0"),
    ("v[0:3]", "v_mfma_f32_16x16x32_bf16 v[16:19], v[8:11], v[12:15], v[2:5]")])
def test_the_reader_finds_every_form(result, reader):
    op = reader.split()[0]
    assert found_in(BF16 % result + "\ts_nop 6\n\t" + reader) == [(op, 7)]
    assert found_in(BF16 % result + "\ts_nop 7\n\t" + reader) == []
    assert found_in(F32 % result + "\ts_nop 7\n\ts_nop 0\n\t" + reader) == [(op, 9)]
    assert found_in(F32 % result + "\ts_nop 7\n\ts_nop 1\n\t" + reader) == []
    # along a taken branch
    assert found_in(BF16 % result + "\ts_cbranch_scc1 .LBB0_1\n\ts_nop 7\n.LBB0_1:\n\t" + reader) == [(op, 1)]


@pytest.mark.parametrize("other", ["v_add_f32_e32 v4, v5, v6", "global_load_dwordx4 v[0:3], v4, s[0:1]", "v_accvgpr_read_b32 v4, a0",
                                   "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]", "ds_read_b128 v[0:3], v4"])
def test_the_reader_passes_what_does_not_wait(other):
    assert found_in(BF16 % "v[0:3]" + "\t" + other) == []


def listing(unit, folder):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    out = os.path.join(folder, unit + ".s")
    subprocess.run([hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", "-I" + CSRC, "--cuda-device-only", "-S", os.path.join(CSRC, unit + ".hip"), "-o", out],
                   check=True, stderr=subprocess.DEVNULL)
    with open(out) as f:
        return f.read()


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    if not shutil.which(os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")):
        pytest.skip("needs hipcc")
    folder = str(tmp_path_factory.mktemp("listings"))
    with concurrent.futures.ThreadPoolExecutor(len(UNITS)) as pool:
        return dict(zip(UNITS, pool.map(lambda u: listing(u, folder), UNITS)))


@pytest.mark.parametrize("unit", UNITS)
def test_results_are_waited_for(listings, unit):
    kernels = functions(listings[unit])
    matrix = sum(op.startswith("v_mfma") for code in kernels.values() for op in code.ops)
    assert matrix > 100 and matrix == len(re.findall(r"^\s+v_mfma", listings[unit], re.M))
    for name, code in kernels.items():
        bad = list(early(code))
        assert not bad, "%s: %s" % (name, bad[:3])
