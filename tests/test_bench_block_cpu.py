"""The committed profiles of the block's operators are of the current sources (CPU only)."""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

BLOCK = os.path.join("grouped_expert_ffn_router_amd", "csrc", "block")


def test_digest_covers_the_sources():
    files = {os.path.join(BLOCK, f) for f in os.listdir(os.path.join(ROOT, BLOCK)) if f.endswith((".hip", ".h"))}
    assert files <= set(bench.BLOCK_SOURCES) and all(os.path.exists(os.path.join(ROOT, p)) for p in bench.BLOCK_SOURCES)
    # headers elsewhere that they include, directly or through another
    seen, todo = set(), [os.path.join(ROOT, f) for f in files]
    while todo:
        p = todo.pop()
        for line in open(p):
            if line.startswith('#include "') and "moe.h" not in line and "entry.hip" not in line:
                q = os.path.normpath(os.path.join(os.path.dirname(p), line.split('"')[1]))
                if q not in seen:
                    seen.add(q)
                    todo.append(q)
    assert {os.path.relpath(q, ROOT) for q in seen} <= set(bench.BLOCK_SOURCES)


def test_committed_profiles_are_of_the_current_sources():
    names = [f for f in os.listdir(os.path.join(ROOT, "profiles")) if f.startswith("block_")]
    assert {"block_kernels_trace.md", "block_pmc.md"} <= set(names)
    for f in names:
        assert bench.source_digest(bench.BLOCK_SOURCES) in open(os.path.join(ROOT, "profiles", f)).read(), f
