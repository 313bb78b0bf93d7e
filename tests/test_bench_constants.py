"""bench.py's constants that were measured on particular kernel sources."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_traffic_was_captured_from_these_sources():
    """Bytes of DRAM traffic per launch are reported while the sources hash to what was profiled; a change of these
    sources asks for a new capture."""
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    import bench
    assert {"prefill", "decode"} <= set(bench.TRAFFIC)
    for name, t in bench.TRAFFIC.items():
        assert bench._src_hash(t["src"]) == t["sha1"], name
