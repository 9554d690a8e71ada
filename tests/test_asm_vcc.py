"""Wait states between a vector instruction that writes VCC and one that reads it, where
inline assembly holds either (CPU: compiles to gfx950 assembly).

gfx950 needs two wait states between a vector ALU instruction that writes VCC (a
compare, an add with carry out) and a vector ALU instruction that reads it (a select,
an add with carry in); the read would see the old mask.  The compiler inserts them
between its own instructions, not inside an inline-asm block or at its edges.
"""
import os
import re
import subprocess

import pytest

from .test_asm_hazards import CSRC, FLAGS, HIPCC, wait_states

# By form: the 32-bit encodings name VCC as their first or last operand.
CARRY = r"v_(add|sub|subrev|addc|subb|subbrev)_co_u32\w*"
WRITES = re.compile(r"v_cmp_\w+|v_div_scale_\w+|" + CARRY)
READS = re.compile(r"v_div_fmas_\w+")


def writes_vcc(line):
    op, _, rest = line.partition(" ")
    at = 0 if op.startswith("v_cmp") else 1  # the mask follows the value in the others
    return bool(WRITES.fullmatch(op)) and "vcc" in (rest.split(",") + [""])[at]


def reads_vcc(line):
    op, _, rest = line.partition(" ")
    if not op.startswith("v_"):
        return False
    if READS.fullmatch(op):
        return True
    return any("vcc" in x for x in rest.split(",")[2 if re.fullmatch(CARRY, op) else 1:])


def stale_vcc(asm):
    """Vector reads of VCC fewer than two wait states after a vector write of it, in program
    order, with the read or the write inside an inline-asm block."""
    found = []
    for func in re.split(r"\n(?=_Z\w+:)", asm):
        name = func.split(":", 1)[0].strip()
        since, wrote_in_asm, in_asm = 2, False, False
        for raw in func.split("\n"):
            line = raw.strip()
            if line.startswith(";;#ASM"):
                in_asm = line.startswith(";;#ASMSTART")
                continue
            if not line or line.startswith((";", ".")) or line.endswith(":"):
                continue
            if since < 2 and reads_vcc(line) and (in_asm or wrote_in_asm):
                found.append((name[:70], line))
            since += wait_states(line)
            if writes_vcc(line):
                since, wrote_in_asm = 0, in_asm
    return found


# Only the tile kernels' assembly names VCC.  It is in every tile alike; these cover both types,
# small and large tiles, and the layouts that use it.
KERNELS = """#include "%s/lm_tile.hpp"
using namespace sgemm::lm;
#define KERNEL(T, LB, RG, EP, ...) template __global__ void sgemm::lm::tile_kernel<T, __VA_ARGS__, KC, LB, RG, EP, true>(TileArgs);
KERNEL(bf16, KC, ROWS, STORE, 16, 64, 1, 4, 4, 16, 4)
KERNEL(bf16, MC, PLAIN, PART, 128, 192, 2, 2, 2, 16, 2)
KERNEL(bf16, KC, PLAIN, GRAD, 256, 256, 2, 2, 2, 32, 1)
KERNEL(float, KC, PLAIN, STATS, 48, 128, 1, 4, 3, 16, 2)
KERNEL(float, MC, ROWS, STORE, 128, 128, 2, 2, 2, 16, 2)
"""


def test_vcc_is_settled_before_inline_asm_reads_it(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    for name in os.listdir(CSRC):
        with open(os.path.join(CSRC, name)) as f:
            assert name == "lm_tile.hpp" or not re.search(r'"[^"\n]*\bvcc\b', f.read()), name
    source, out = tmp_path / "tiles.hip", tmp_path / "tiles.s"
    source.write_text(KERNELS % CSRC)
    subprocess.run([HIPCC, *FLAGS, "-o", str(out), str(source)], check=True, stderr=subprocess.DEVNULL)
    asm = out.read_text()
    assert asm.count("v_cndmask_b32") and len(re.findall(r"^_Z\w+:", asm, re.M)) == 5
    found = stale_vcc(asm)
    assert not found, "%d reads of VCC too soon after its write: %s" % (len(found), found[:3])


def test_scanner_finds_stale_vcc():
    """The scanner itself: one wait state is too few, two are enough, and what the compiler
    placed outside the blocks is left to it."""
    def kernel(gap, inside=True):
        marks = [";;#ASMSTART", ";;#ASMEND"] if inside else ["; start", "; end"]
        return "\n".join(["_Zk:", marks[0], "v_cmp_gt_i32_e32 vcc, s3, v2", *gap,
                          "v_cndmask_b32_e32 v1, v4, v1, vcc", marks[1]])
    assert stale_vcc(kernel([])) and stale_vcc(kernel(["s_nop 0"]))
    assert not stale_vcc(kernel(["s_nop 1"])) and not stale_vcc(kernel([], inside=False))
    edge = "\n".join(["_Zk:", "v_cmp_gt_i32_e32 vcc, s3, v2", ";;#ASMSTART",
                      "v_cndmask_b32_e32 v1, v4, v1, vcc", ";;#ASMEND"])
    assert stale_vcc(edge)
