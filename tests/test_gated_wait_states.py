"""Wait states of the gated product's loads into LDS, in the assembly that the compiler
makes of it (no GPU).

The loads are written as inline assembly, in front of which the compiler puts no wait
states of its own.  A vector instruction that writes a scalar register (a value made
uniform, a spilled one read back) has to be 5 wait states ahead of a memory instruction
that reads it; every instruction between is one, s_nop n is n + 1.  Scalar instructions'
results are waited for by the hardware."""
import os
import re
import subprocess

import pytest

from level_haar_wavelet_amd import build

STATES = 5


def scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"s(\d+)$", operand)
    return {int(m[1])} if m else set()


def instructions(lines):
    """(name, operands) of the instructions; labels and directives apart."""
    for line in lines:
        text = line.split(";")[0].strip()
        if not text or text.startswith(".") or text.endswith(":"):
            continue
        name, _, rest = text.partition(" " if " " in text else "\t")
        yield name, [q for part in rest.replace("\t", " ").split(",") for q in part.split()]


def close_pairs(lines):
    """(loads into LDS, those that read a scalar register too soon)."""
    written, loads, bad = [], 0, []  # what the last instructions wrote, and their wait states
    for name, operands in instructions(lines):
        if name.startswith("buffer_load") and "lds" in operands:
            loads += 1
            reads = set().union(*map(scalars, operands))
            states = 0
            for what, n in reversed(written):
                if states >= STATES:
                    break
                if what & reads:
                    bad.append((name, operands))
                    break
                states += n
        # a vector instruction's result comes first, a carry or a condition second
        writes = set().union(*map(scalars, operands[:2])) if name.startswith("v_") else set()
        written.append((writes, int(operands[0], 0) + 1 if name == "s_nop" else 1))
        del written[:-STATES]
    return loads, bad


def test_the_check_itself():
    load = "\tbuffer_load_dwordx4 v1, s[4:7], s8 offen lds"
    for first in ("\tv_readfirstlane_b32 s5, v0", "\tv_readlane_b32 s8, v0, 3", "\tv_add_co_u32_e64 v1, s[6:7], v2, v3"):
        for between, states in (([], 0), (["\ts_mov_b32 m0, s9", "\ts_nop 0"], 2), (["\ts_nop 3"], 4), (["\ts_nop 4"], 5),
                                (["\ts_mov_b32 m0, s9", "\ts_nop 3"], 5), (["\tv_mov_b32 v5, v6"] * 5, 5)):
            loads, bad = close_pairs([first] + between + [load])
            assert loads == 1 and bool(bad) == (states < STATES)
    assert close_pairs(["\ts_mov_b32 s5, s1", load]) == (1, [])
    assert close_pairs(["\tv_readfirstlane_b32 s9, v0", load, "\tbuffer_load_dword v1, v2, s[4:7], 0 offen"]) == (1, [])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_loads_into_lds(dtype, tmp_path):
    out = tmp_path / "gated.s"
    cmd = [build.HIPCC] + build.FLAGS + ["-w", "--offload-device-only", "-S", "-o", str(out),
                                         os.path.join(build.TRAIN, "wtconv_gated_%s.hip" % dtype)]
    subprocess.run(cmd, check=True, capture_output=True, timeout=600)
    with open(out) as lines:
        loads, bad = close_pairs(lines)
    assert loads > 100 and not bad, bad[:5]
