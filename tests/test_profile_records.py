"""The committed traffic records hold for the kernels' sources as they are."""
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["score_sp_traffic.json", "decode_split_traffic.json"])
def test_traffic_records_match_the_sources(name):
    """bench.py reports no traffic for a kernel whose sources changed since its record was taken: a change to one of
    them, or to a header that they share, brings a record of its own."""
    import bench
    with open(os.path.join(ROOT, "profiles", name)) as f:
        assert bench.traffic_record(name) == json.load(f)
