"""The wait states that hand-written assembly owes the hardware, in the compiler's assembly of every source that has
such loads (mfma.h). Nothing checks these on the chip, and the compiler keeps them for its own instructions alone:

* a vector-memory instruction reads a scalar register that a vector instruction (v_readfirstlane, v_readlane, ..) wrote
  five wait states after the write at the earliest;
* a load into LDS reads m0 one wait state after its change at the earliest.

An instruction is one wait state, s_nop n is n + 1."""

import os
import re
import subprocess

import pytest

from packed_varlen_gated_amd import build

SOURCES = ["attn_fwd.hip", "attn_paged.hip", "attn_window_bwd.hip"]


def test_every_source_with_such_loads_is_looked_at():
    text = {f: open(os.path.join(build.CSRC, f)).read() for f in os.listdir(build.CSRC)}
    asm = r"asm\s+volatile\s*\(\s*[^\"\s]|asm\s+volatile\s*\(\s*\"[^\"]"     # with instructions in it
    assert {f for f in text if re.search(asm, text[f])} == {"mfma.h"}
    assert {f for f in text if f.endswith(".hip") and "_async" in text[f]} == set(SOURCES)


def assembly(source, tmp):
    out = os.path.join(str(tmp), source + ".s")
    r = subprocess.run([build.HIPCC] + build.COMMON_FLAGS + ["--offload-device-only", "-S",
                       os.path.join(build.CSRC, source), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return open(out).read()


def _scalars(operand):
    """The scalar registers that an operand names."""
    m = re.fullmatch(r"s(\d+)", operand) or re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[m.lastindex]) + 1))
    return {operand} if operand in ("vcc", "m0") else set()


def late_loads(text):
    """(loads into LDS in hand-written blocks, [(line, what is missing)])."""
    before, found, bad = [], 0, []         # instructions of the kernel so far: (states, name, operands)
    block = -1                             # where the hand-written block began
    for number, line in enumerate(text.splitlines(), 1):
        line = line.split("//")[0].strip()
        if line.endswith("#ASMSTART"):
            block = len(before)
        elif line.endswith("#ASMEND"):
            block = -1
        if not line or line[0] in ".;_" or line.endswith(":"):
            continue
        name, _, rest = line.partition(" ")
        ops = [x.strip() for x in rest.split(";")[0].split(",")]
        if name.startswith("buffer_load") and rest.split()[-1] == "lds":
            reads = set().union(*(_scalars(x.split()[0]) for x in ops))
            states, own = 0, block >= 0 and not any(x[1].startswith("buffer") for x in before[block:])
            found += block >= 0
            if own and sum(x[0] for x in before[block:]) < 5:
                bad.append((number, "wait states of the block's own before its first load"))
            for n, was, to in reversed(before):
                if states < 1 and was.startswith("s_") and to[0] == "m0":
                    bad.append((number, "m0"))
                if was.startswith("v_") and _scalars(to[0]) & reads:
                    bad.append((number, f"{was} {to[0]}, {states} wait states"))
                states += n
                if states >= 5:
                    break
        before.append((int(ops[0], 0) + 1 if name == "s_nop" else 1, name, ops))
    return found, bad


def test_the_check_sees_what_is_missing():
    """On texts whose faults are known."""
    block = lambda nop: f""";;#ASMSTART
	s_mov_b32 s3, m0
	s_mov_b32 m0, s83
	s_nop {nop}
	buffer_load_dwordx4 v2, s[8:11], 0 offen lds
	s_add_u32 m0, m0, 0x1000
	s_nop 0
	buffer_load_dwordx4 v3, s[8:11], 0 offen lds
	s_mov_b32 m0, s3
	;;#ASMEND
"""
    for write in ("v_readfirstlane_b32 s10, v23", "v_readlane_b32 s11, v1, 4", "v_cmp_eq_u32_e64 s[8:9], v0, v1"):
        assert late_loads(f"\t{write}\n\t" + block(2)) == (2, [])
        found, bad = late_loads(f"\t{write}\n\t" + block(0))
        assert found == 2 and len(bad) == 2 and bad[1][1].endswith("3 wait states")
    assert late_loads("\tv_readfirstlane_b32 s12, v23\n\t" + block(2)) == (2, [])
    assert [b[1] for b in late_loads(block(2).replace("s_nop 0\n\t", ""))[1]] == ["m0"]


@pytest.mark.parametrize("source", SOURCES)
def test_loads_into_lds_wait_for_their_scalars(source, tmp_path):
    found, bad = late_loads(assembly(source, tmp_path))
    assert found > 20
    assert bad == []
