"""The products' kernels as the compiler leaves them (gfx950 assembly, no GPU).

A matrix instruction's result is there some cycles after it is issued, and
nothing in the hardware holds another instruction back that touches the
result's registers before: the compiler has to put waits between.  So every
matrix instruction has to be one that the compiler knows, and its accumulators
have to stay in place in the loops (a move of them there would be such a
touch, and costs as much as it moves)."""
import os
import re
import subprocess

import pytest

from lossless_bf16_exponent_zc_amd import build

SOURCE = os.path.join(build.CSRC, "zc_product.hip")
# 8 passes of 4 cycles, after which the result may be read: the wait of the
# compiler's own in kernels whose results are read at once
WAITS = 12


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "zc_product.s")
    cmd = [build.HIPCC, *build.FLAGS, "-Wno-unused-command-line-argument", "-S", "--cuda-device-only", SOURCE, "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found, lines = {}, None
    for line in open(out):
        name = re.match(r"(_Z\w+):", line)
        if name:
            lines = found.setdefault(name.group(1), [])
        elif line.startswith(".Lfunc_end"):
            lines = None
        elif lines is not None and re.match(r"\s+[a-z]|\.LBB", line):
            lines.append(line.strip())
    found = {k: v for k, v in found.items() if any("v_mfma" in x for x in v)}
    assert len(found) == 30  # five products and five weight gradients, of three types
    return found


def registers(text):
    got = set()
    for kind, lo, hi in re.findall(r"\b([av])\[(\d+):(\d+)\]", text):
        got |= {(kind, i) for i in range(int(lo), int(hi) + 1)}
    return got | {(kind, int(i)) for kind, i in re.findall(r"\b([av])(\d+)\b", text)}


def inner_loops(lines):
    label = {x.split(":")[0]: i for i, x in enumerate(lines) if x.startswith(".LBB")}
    spans = []
    for i, x in enumerate(lines):
        m = re.match(r"s_c?branch\S*\s+(\.LBB\w+)", x)
        if m and label.get(m.group(1), i) < i:
            spans.append((label[m.group(1)], i))
    return [lines[a:b] for a, b in spans if not any(a <= c and d <= b and (a, b) != (c, d) for c, d in spans)]


def test_the_compiler_knows_every_matrix_instruction():
    """None stands in inline assembly, whose registers it does not wait for."""
    for f in os.listdir(build.CSRC):
        text = open(os.path.join(build.CSRC, f)).read()
        for asm in re.findall(r"\basm\b.*?;", text, re.S):
            assert "mfma" not in asm, (f, asm)


def test_accumulators_stay_in_place_in_the_loops(kernels):
    for name, lines in kernels.items():
        for loop in inner_loops(lines):
            if any("v_mfma" in x for x in loop):
                assert not any("v_accvgpr" in x for x in loop), name
                assert not any("scratch_" in x for x in loop), name


def test_waits_before_results_are_touched(kernels):
    """Straight on from every matrix instruction: whatever else names its
    result comes after the wait."""
    for name, lines in kernels.items():
        recent = []  # [waits since, registers]
        for x in lines:
            op = x.split()[0]
            if op in ("s_branch", "s_endpgm"):
                recent = []
            elif x.startswith(".LBB"):
                continue
            elif op.startswith("v_mfma"):
                recent = [[n + 1, r] for n, r in recent if n < 64] + [[0, registers(x.split(",")[0])]]
            else:
                used = registers(x)
                for n, r in recent:
                    assert n >= WAITS or not used & r, (name, x)
                step = 1 + int(x.split()[1]) if op == "s_nop" else 1
                recent = [[n + step, r] for n, r in recent if n + step < 64]
