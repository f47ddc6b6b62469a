"""The recorded DRAM traffic of the bench's kernels is of the sources that are there: a change of one
of a kernel's sources needs the record taken again."""
import json
import os

import pytest

import bench

RECORD = json.load(open(os.path.join(bench.ROOT, "profiles", "traffic.json")))["entries"]


@pytest.mark.parametrize("entry", RECORD, ids=lambda e: e["workload"])
def test_the_record_is_current(entry):
    assert bench.recorded_traffic(entry["kernel"], entry["workload"]) == entry["bytes_per_launch"]
