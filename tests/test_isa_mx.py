"""Static check of the hand-issued LDS reads of the MX-FP4 product (CPU only).

The same walk as for the bf16 core (test_isa_lds_reads.py): no instruction
may touch the destination of an inline LDS read before an s_waitcnt retires
it.  The MX-FP4 kernel also reads its scales that way, 4 bytes at a time
(ds_read_b32); the walk tracks destinations whatever their width.
"""

import os
import re
import shutil
import subprocess
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_isa_lds_reads as isa  # noqa: E402

OPS = os.path.join(isa.CSRC, "ops")
ALLOWED = ("ds_read_b128", "ds_read_b32", "s_waitcnt", "s_barrier")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if not (os.path.exists(isa.HIPCC) or shutil.which(isa.HIPCC)):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa_mx") / "mx.s"
    cmd = [isa.HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "--cuda-device-only", "-S",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(isa.ROOT, "include"), "-I", isa.CSRC, os.path.join(OPS, "mx.hip"), "-o", str(out)]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-3000:]
    return out.read_text()


def _tile_kernels(asm):
    lines = asm.split("\n")
    for s in (i for i, l in enumerate(lines) if re.match(r"^_Z\w*mx_gemm_tile\w*:", l)):
        e = next(i for i in range(s, len(lines)) if lines[i].startswith(".Lfunc_end"))
        yield lines[s].rstrip(":"), lines[s:e]


def _as_tracked(body):
    """Inline ds_read_b32 spelled as the read that the walk tracks."""
    out, in_asm = [], False
    for l in body:
        in_asm = True if l.strip().startswith(";;#ASMSTART") else False if l.strip().startswith(";;#ASMEND") else in_asm
        out.append(l.replace("ds_read_b32 ", "ds_read_b128 ") if in_asm else l)
    return out


def test_no_instruction_touches_a_read_in_flight(asm):
    kernels = list(_tile_kernels(asm))
    assert len(kernels) >= 5
    for name, body in kernels:
        assert sum("ds_read_b32 " in l for l in body) > 0 and sum("ds_read_b128 " in l for l in body) > 0, name
        bad = isa._violations(_as_tracked(body))
        assert not bad, f"{name}: {len(bad)} hazards, first: {bad[:3]}"


def test_the_walk_sees_a_planted_scale_read():
    body = [";;#ASMSTART", "ds_read_b32 v10, v2", ";;#ASMEND", "v_mov_b32_e32 v20, v10",
            ";;#ASMSTART", "s_waitcnt lgkmcnt(0)", ";;#ASMEND"]
    assert isa._violations(_as_tracked(body))


def test_inline_assembly_is_only_lds_reads_waits_and_barriers(asm):
    bad = [(fn, line) for fn, line in isa._asm_blocks(asm) if not line.split()[0].startswith(ALLOWED)]
    assert not bad, bad[:3]


def test_operator_sources_hold_no_other_inline_assembly():
    for fname in sorted(os.listdir(OPS)):
        src = open(os.path.join(OPS, fname)).read()
        assert len(re.findall(r"\basm\b\s*(volatile)?\s*\(", src)) == len(re.findall(r"\basm volatile\(\"", src)), fname
        for m in re.finditer(r"\basm\s+volatile\s*\(\s*\"([^\"]*)\"", src):
            assert m.group(1).split()[0].startswith(ALLOWED), f"{fname}: {m.group(1)}"
