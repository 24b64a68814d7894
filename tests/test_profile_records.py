"""The committed counter record that bench.py reports belongs to the Hessian's current source."""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def test_hessian_traffic_is_of_the_current_source():
    import bench
    # a stale record is silently left out of the benchmark's line
    for workload in ("mlp_down_28672", "attn_4096"):
        assert bench.load_traffic(workload), f"retake the counters of {workload}"
