"""The DRAM bytes that the bench reports beside its rates: each record is of the sources that are
there, or the bench leaves it out."""
import json
import os

import pytest

import bench

RECORDS = json.load(open(os.path.join(bench.ROOT, "profiles", "ncu_traffic.json")))


@pytest.mark.parametrize("name", sorted(RECORDS))
def test_the_record_is_of_the_present_sources(name):
    kernel = name.removesuffix("_small")
    assert RECORDS[name]["source_sha"] == bench.kernel_source_sha(kernel)
