"""The committed traffic records belong to the committed kernels: the bench
drops a record whose sources changed, and its roofline then names no traffic."""
import glob
import os

import pytest

import bench

RECORDS = sorted(os.path.basename(p) for p in glob.glob(os.path.join(bench.ROOT, "profiles", "*_traffic.json")))


@pytest.mark.parametrize("name", RECORDS)
def test_record_is_of_these_sources(name):
    assert bench._traffic_record(name) is not None, f"profiles/{name}: its sources changed, take it again"
