"""The recorded DRAM traffic of the headline kernel holds for its present
sources, so the bench reports it."""
import json

import bench


def test_recorded_traffic_is_of_the_present_sources():
    with open(bench.TRAFFIC_FILE) as f:
        record = json.load(f)
    assert record
    for key, e in record.items():
        kernel, workload = key.split("@")
        assert bench.profiled_traffic(kernel, workload) == e["bytes_per_launch"], e["sources"]
