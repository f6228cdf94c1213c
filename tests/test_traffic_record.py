"""The HBM counters on record are those of the linears' present source."""
import json
import os

import bench


def test_traffic_of_every_recorded_launch_is_reported():
    with open(os.path.join(bench.ROOT, "profiles", "hbm_traffic.txt")) as f:
        entries = json.load(f)["entries"]
    assert entries
    for key, entry in entries.items():
        workload, m = key.rsplit("/M", 1)
        assert bench.measured_traffic(workload, int(m)) == entry["traffic_bytes_per_launch"], key
