"""The DRAM traffic that bench.py reports is of the kernels as they are: it drops a figure whose sources have changed, so a change
of theirs needs a new measurement (the command is beside the figure)."""
import json
import os

import pytest

import bench


@pytest.mark.parametrize("name", sorted(bench.KERNEL_SOURCES))
def test_recorded_traffic_is_of_these_sources(name):
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        record = json.load(f)[name]
    assert record["source_sha256_16"] == bench._source_hash(bench.KERNEL_SOURCES[name])
    assert record["dram_bytes_per_launch"] > 0
