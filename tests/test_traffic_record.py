"""The recorded DRAM traffic of the attention kernels belongs to the sources as they are."""
import json
import os

import bench


def test_traffic_record_is_of_the_present_attention_source():
    with open(os.path.join(bench.ROOT, "profiles", "attend_traffic.json")) as f:
        for name in json.load(f):
            assert bench.traffic_from_profile(name), f"profiles/attend_traffic.json: {name} is stale"
