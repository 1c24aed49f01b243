"""The DRAM traffic that the bench reports comes from recorded counters, and is null where a kernel's sources
have changed since: a change beside those kernels is not to touch their files."""
import json
import os

import bench


def test_recorded_traffic_holds_for_the_sources():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        entries = json.load(f)
    assert entries
    for kernel, entry in entries.items():
        assert bench.committed_traffic(kernel) == entry["bytes_per_launch"], kernel
