"""Wait states in front of the asm loads to LDS, read from the assembly that
the compiler makes of this repository's kernels (no GPU needed).

A scalar register that the vector ALU has written may be read by a
vector-memory instruction five wait states later (an instruction is one,
s_nop n is n + 1). The compiler keeps to that for its own instructions but not
inside asm, so the loads have to bring the five themselves, whatever stands in
front of them."""
import os
import re
import subprocess

import pytest

from block_scaled_bit_quantize_amd import build as B

NEEDED = 5


def scalars(operand):
    """The scalar registers of an operand: s7, s[4:7]."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m[1])} if m else set()


def faults(text):
    """(loads to LDS, those that may come too soon after a vector ALU's write of a register they read). A label within
    the five counts as such a write: what comes before the load is then not known."""
    loads, bad, seen = 0, [], []
    for number, line in enumerate(text.splitlines(), 1):
        code = line.split(";")[0].strip()
        if not code or (code.startswith(".") and not code.endswith(":")):
            continue
        if code.endswith(":"):
            seen.append((None, [], 0))
            continue
        op, _, rest = code.partition(" ")
        args = [a.strip() for a in rest.split(",")]
        if op.startswith("buffer_load") and code.split()[-1] == "lds":
            loads += 1
            reads = set().union(*(scalars(a.split()[0]) for a in args if a))
            states = 0
            for o, a, cost in reversed(seen):
                if states >= NEEDED:
                    break
                if o is None or (o.startswith("v_") and scalars(a[0]) & reads):
                    bad.append((number, states, o))
                    break
                states += cost
        seen = seen[-31:] + [(op, args, int(args[0], 0) + 1 if op == "s_nop" else 1)]
    return loads, bad


@pytest.mark.parametrize("text,n", [
    ("v_readlane_b32 s5, v1, s2\ns_mov_b32 m0, s9\ns_nop 0\nbuffer_load_dword v1, s[4:7], s8 offen lds", 1),
    ("v_readlane_b32 s5, v1, s2\ns_mov_b32 m0, s9\ns_nop 3\nbuffer_load_dword v1, s[4:7], s8 offen lds", 0),
    ("v_readlane_b32 s3, v1, s2\ns_mov_b32 m0, s9\ns_nop 0\nv_mov_b32 v1, v2\ns_nop 0\ns_nop 0\n"
     "buffer_load_dword v1, s[4:7], s8 offen lds", 0),
    (".LBB0_1:\ns_mov_b32 m0, s9\ns_nop 0\nbuffer_load_dword v1, s[4:7], s8 offen lds", 1),
])
def test_the_reader(text, n):
    loads, bad = faults(text)
    assert loads == 1 and len(bad) == n


@pytest.mark.parametrize("source", ["moe_few.hip", "int8.hip"])
def test_loads_to_lds_wait_for_their_scalars(source, tmp_path):
    out = str(tmp_path / "k.s")
    r = subprocess.run([B.HIPCC, *B.FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, source), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    loads, bad = faults(open(out).read())
    assert loads > 100
    assert not bad, f"{len(bad)} of {loads} loads, the first (line, wait states, instruction): {bad[:5]}"
