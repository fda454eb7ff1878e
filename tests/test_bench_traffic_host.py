"""bench.py's lines state the DRAM bytes of a call only where they were recorded on the current kernel sources."""
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

with open(os.path.join(ROOT, "profiles", "dram_traffic.json")) as f:
    RECORDED = json.load(f)


@pytest.mark.parametrize("key", sorted(RECORDED))
def test_the_record_is_of_the_current_sources(key):
    assert bench.recorded_traffic(key) == RECORDED[key]["bytes_per_launch"] > 0


def test_the_record_tells_sources_of_other_kernels_apart():
    """What the bench's workloads launch is hashed; sources of the cache's kernels may change under the record."""
    names = [n for n in os.listdir(os.path.join(ROOT, "skinny_gemm_bit_gb300", "csrc")) if n.endswith((".cu", ".cuh", ".h"))]
    left_out = {n for n in names if n.startswith(bench.OTHER_SOURCES)}
    assert "tfq_cache.h" in left_out and "tfq_ptx.cuh" not in left_out and "tfq_qproj.cuh" not in left_out
