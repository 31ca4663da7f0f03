"""The DRAM traffic that bench.py reports comes from recorded captures, which
count only for the kernel sources they were taken on: each record in the
repository is one that bench.py still takes."""
import json
import os

import pytest

import bench


@pytest.mark.parametrize("kind", ["decode", "prefill", "grouped"])
def test_the_recorded_capture_belongs_to_the_current_sources(kind):
    with open(os.path.join(bench.ROOT, "profiles", f"{kind}_traffic.json")) as f:
        rec = json.load(f)
    got = bench._recorded_traffic(rec["workload"], rec.get("launch", "pa_decode"), kind)
    assert got == rec["dram_bytes_per_launch"] and got
