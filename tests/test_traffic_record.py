"""profiles/traffic.json belongs to the kernels that are there: bench.py reports a
recorded DRAM traffic only while the partial kernels' sources are those it was
captured from, so a change to them wants a new capture."""
import json
import os

import pytest

import bench

with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
    RECORDED = sorted(k for k in json.load(f) if not k.startswith("_"))


def test_there_are_records():
    assert "llama8b" in RECORDED


@pytest.mark.parametrize("name", RECORDED)
def test_captured_from_these_sources(name):
    assert bench.recorded_traffic(name) is not None, bench.kernel_source_hash()
