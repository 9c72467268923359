"""The DRAM-traffic ratios on file belong to the kernels as they are: a change of a captured kernel's sources
needs a new capture (or the entry's removal), else bench.py reports no traffic for it."""
import json

import bench


def test_every_traffic_ratio_is_of_the_present_sources():
    with open(bench.TRAFFIC_FILE) as f:
        entries = json.load(f)["entries"]
    assert entries
    for e in entries:
        assert bench.source_digest(e["sources"]) == e["sources"], e["kernel"]
        ratio, note = bench.traffic_ratio(e["kernel"], e["latent"])
        assert ratio == e["ratio"], note
