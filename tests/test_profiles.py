"""The DRAM figures that bench.py reports beside its own timings were taken on
the kernel sources that are committed: a figure of older sources is taken again
or leaves the file."""
import json
import os

import bench


def test_traffic_was_taken_on_these_sources():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        entries = {k: v for k, v in json.load(f).items() if not k.startswith("_")}
    assert entries
    for key, entry in entries.items():
        workload, stage = key.split(":")
        assert bench.ncu_traffic(stage, workload) == entry["dram_bytes_per_launch"], key
