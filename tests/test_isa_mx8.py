"""Static check of the hand-issued LDS reads of the MX-FP8 by MX-FP4 product (CPU only): the walk of
test_isa_lds_reads.py over its tile kernels, and no other inline assembly in the operators' sources."""

import os
import re
import shutil
import subprocess
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_isa_lds_reads as isa  # noqa: E402
import test_isa_mx as mx  # noqa: E402

BLOCK = os.path.join(isa.CSRC, "block")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if not (os.path.exists(isa.HIPCC) or shutil.which(isa.HIPCC)):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa_mx8") / "mx8.s"
    cmd = [isa.HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "--cuda-device-only", "-S",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(isa.ROOT, "include"), "-I", isa.CSRC, os.path.join(BLOCK, "mx8_gemm.hip"), "-o", str(out)]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-3000:]
    return out.read_text()


def test_no_instruction_touches_a_read_in_flight(asm):
    lines = asm.split("\n")
    starts = [i for i, l in enumerate(lines) if re.match(r"^_Z\w*mx8_gemm_tile\w*:", l)]
    assert len(starts) >= 3
    for s in starts:
        body = lines[s:next(i for i in range(s, len(lines)) if lines[i].startswith(".Lfunc_end"))]
        assert sum("ds_read_b32 " in l for l in body) > 0 and sum("ds_read_b128 " in l for l in body) > 0
        bad = isa._violations(mx._as_tracked(body))
        assert not bad, f"{lines[s]}: {len(bad)} hazards, first: {bad[:3]}"


def test_the_matrix_instructions_stay_between_the_reads(asm):
    """No more than one substep's matrix instructions (8) come without a read, load, wait or branch among them: the compiler
    has not gathered those of a whole step in one place."""
    lines = asm.split("\n")
    for s in (i for i, l in enumerate(lines) if re.match(r"^_Z\w*mx8_gemm_tile\w*:", l)):
        run = longest = 0
        for l in lines[s:next(i for i in range(s, len(lines)) if lines[i].startswith(".Lfunc_end"))]:
            run = run + 1 if "v_mfma" in l else 0 if re.match(r"\s+(ds_read|global_load_lds|s_barrier|s_cbranch|s_waitcnt)", l) else run
            longest = max(longest, run)
        assert longest <= 8, (lines[s], longest)


def test_inline_assembly_is_only_lds_reads_waits_and_barriers(asm):
    bad = [(fn, line) for fn, line in isa._asm_blocks(asm) if not line.split()[0].startswith(mx.ALLOWED)]
    assert not bad, bad[:3]


def test_block_sources_hold_no_other_inline_assembly():
    for fname in sorted(os.listdir(BLOCK)):
        src = open(os.path.join(BLOCK, fname)).read()
        assert len(re.findall(r"\basm\b\s*(volatile)?\s*\(", src)) == len(re.findall(r"\basm volatile\(\"", src)), fname
        for m in re.finditer(r"\basm\s+volatile\s*\(\s*\"([^\"]*)\"", src):
            assert m.group(1).split()[0].startswith(mx.ALLOWED), f"{fname}: {m.group(1)}"
