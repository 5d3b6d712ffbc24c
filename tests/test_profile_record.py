"""The committed traffic records of the expert kernel belong to the code that
is here, so that the benchmark's line can quote them."""
import json
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_traffic_records_are_of_this_code():
    with open(os.path.join(ROOT, "profiles", "expert_kernel_traffic.json")) as f:
        records = {k: v for k, v in json.load(f).items() if not k.startswith("_")}
    assert records
    for name, rec in records.items():
        workload, run = name.split("/")
        got = bench.recorded_traffic(workload, run, rec["algorithmic_bytes"])
        assert got is not None and abs(got - rec["dram_bytes"]) <= 1, name
