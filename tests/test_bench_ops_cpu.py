"""Host logic of bench.py for layers with MX-FP4 experts (CPU only)."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402
from workload import configs  # noqa: E402

OPS = os.path.join("grouped_expert_ffn_router_amd", "csrc", "ops")


def test_algorithmic_work_of_the_mx_kernels():
    """Config 3, 22,648 kept rows a wave: the products' operations are those of the bf16 experts; the gather reads rows of
    6144 B, writes 3072 codes and 96 scales of them in 1632 B, and reads a 4-byte place."""
    w = bench.algorithmic_work(configs.get(3), [67944 / 3] * 3, send_kept=65536, send_cap=1127)
    assert w["mx_gate_up"] == w["expert_gate_up"] and w["mx_down"] == w["expert_down"]
    assert w["mx_gather"] == ("byte", 22648 * (6144 + 1632 + 4))
    assert bench.flop_peak("mx_down") == 4 * bench.flop_peak("expert_down") == 10000


def test_operator_digest_covers_the_operators_sources_and_is_not_the_layers():
    files = {os.path.join(OPS, f) for f in os.listdir(os.path.join(ROOT, OPS)) if f.endswith((".hip", ".h"))}
    assert files <= set(bench.OPERATOR_SOURCES) and all(os.path.exists(os.path.join(ROOT, p)) for p in bench.OPERATOR_SOURCES)
    # headers outside ops/ that an operator's source includes, directly or through another
    seen, todo = set(), [os.path.join(ROOT, f) for f in files]
    while todo:
        p = todo.pop()
        for line in open(p):
            if line.startswith('#include "') and "moe.h" not in line and "api.hip" not in line:
                q = os.path.normpath(os.path.join(os.path.dirname(p), line.split('"')[1]))
                if q not in seen:
                    seen.add(q)
                    todo.append(q)
    assert {os.path.relpath(q, ROOT) for q in seen} <= set(bench.OPERATOR_SOURCES)
    assert bench.source_digest(bench.OPERATOR_SOURCES) != bench.source_digest()


@pytest.mark.parametrize("args", [["--config", "2"], ["--sweep-capacity"], ["--dropless"], ["--vendor-gemm"]])
def test_mx_experts_go_with_the_benchmark_line_only(args):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--experts", "mx", *args], stdout=subprocess.PIPE,
                       stderr=subprocess.PIPE, text=True, timeout=300, cwd=ROOT)
    assert r.returncode != 0 and "--experts mx" in r.stderr


def test_committed_operator_profiles_are_of_the_current_sources():
    """Kernel times and counters of the operators, and of the layer with MX-FP4 experts, carry the digest of the sources
    they were taken from."""
    names = [f for f in os.listdir(os.path.join(ROOT, "profiles")) if f.startswith("operators_")]
    assert {"operators_kernels_trace.md", "operators_pmc.md", "operators_mx_layer_cfg3_full_layer_4k.md"} <= set(names)
    for f in names:
        assert bench.source_digest(bench.OPERATOR_SOURCES) in open(os.path.join(ROOT, "profiles", f)).read(), f
