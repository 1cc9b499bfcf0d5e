"""Wait states around inline assembly (CPU: compiles, runs nothing).

gfx9 needs five wait states between a vector instruction that writes a scalar
register (v_readfirstlane, v_readlane) and a vector memory instruction that
reads it; an instruction is one, s_nop N is N + 1. The compiler sees to that
for its own memory instructions but not inside asm blocks, so the generated
assembly is checked: counted back from every such instruction of an asm block,
no vector instruction writes one of its scalar registers within five states,
on any path (a label before them counts as unknown, so as a failure)."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from combine_get_dispatch_counts_amd import build

STATES = 5


def scalars(text: str) -> set[int]:
    """Numbers of the scalar registers named in an instruction's operands."""
    regs = {int(r) for r in re.findall(r"\bs(\d+)\b", text)}
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        regs |= set(range(int(a), int(b) + 1))
    return regs


def written(line: str) -> set[int]:
    """Scalar registers an instruction writes: its first operand, and the
    second where that is a scalar destination too (carries, v_div_scale)."""
    ops = line.split(None, 1)[1] if " " in line or "\t" in line else ""
    first = ops.split(",")
    out = scalars(first[0]) if first else set()
    if len(first) > 1 and re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co|v_div_scale|v_mad_[iu]64",
                                   line):
        out |= scalars(first[1])
    return out


def too_close(lines: list[str]) -> list[str]:
    """Findings in a listing: asm blocks' memory instructions that follow a
    vector write of one of their scalar registers by fewer than STATES."""
    found, inside = [], False
    for i, line in enumerate(lines):
        if ";#ASMSTART" in line or ";#ASMEND" in line:
            inside = "ASMSTART" in line
            continue
        s = line.split(";")[0].strip()
        if not inside or not re.match(r"(buffer|global|flat|scratch)_", s):
            continue
        need, states, j = scalars(s.split(None, 1)[1]), 0, i - 1
        while states < STATES and j >= 0:
            p = lines[j].split(";")[0].strip()
            j -= 1
            if not p or (p.startswith(".") and not p.endswith(":")):
                continue
            if p.endswith(":"):
                found.append(f"line {i + 1}: {s}: {states} states behind {p}")
                break
            if p.startswith("v_") and written(p) & need:
                found.append(f"line {i + 1}: {s}: {states} states behind {p}")
                break
            if p.startswith("s_") and not re.match(r"s_(cmp|bitcmp)", p):
                need = need - written(p)     # a scalar instruction's result is waited for
            states += int(p.split()[1], 0) + 1 if p.startswith("s_nop") else 1
    return found


def test_the_check_itself():
    block = [";;#ASMSTART", "s_mov_b32 m0, s0", "s_nop %d",
             "buffer_load_dwordx4 v1, s[4:7], s9 offen lds", ";;#ASMEND"]

    def listing(before, nop):
        return ["f:"] + ["v_mov_b32 v0, v1"] * 6 + before + [b % nop if "%" in b else b for b in block]

    assert too_close(listing(["v_readfirstlane_b32 s6, v2"], 0))
    assert too_close(listing(["v_readlane_b32 s9, v2, 3"], 2))
    assert not too_close(listing(["v_readfirstlane_b32 s6, v2"], 3))
    assert not too_close(listing(["v_readfirstlane_b32 s8, v2"], 0))
    assert not too_close(listing(["v_readfirstlane_b32 s6, v2"] + ["v_mov_b32 v0, v1"] * 3, 0))
    assert too_close(listing([".LBB0_1:"], 0))
    assert not too_close(listing(["v_readlane_b32 s9, v2, 3", "s_lshl_b32 s9, s9, 2"], 0))
    assert too_close(listing(["v_add_co_u32_e64 v3, s[4:5], v1, v2"], 0))


@pytest.mark.parametrize("src", [s for s in build.SOURCES
                                 if re.search(r"\basm\b", open(os.path.join(build.CSRC, s)).read())])
def test_asm_memory_instructions(src, tmp_path):
    out = str(tmp_path / "listing.s")
    r = subprocess.run([build.hipcc(), *build.flags(), "--offload-device-only", "-S",
                        os.path.join(build.CSRC, src), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lines = open(out).read().splitlines()
    if src == "grouped.hip":
        assert sum("buffer_load_dwordx4" in v and v.rstrip().endswith("lds") for v in lines) > 100
    found = too_close(lines)
    assert not found, f"{len(found)} of {src}, first: {found[0]}"
