"""The DRAM-traffic records stand for the kernels as they are: a change of a row's
sources takes a new capture with it, and what is not a row's kernel stays out of the
files that are hashed for it.  No GPU."""
import pytest

import bench


@pytest.mark.parametrize("row", bench.ROWS)
def test_every_record_is_of_the_present_sources(row):
    assert bench.traffic_records()[row]["sources"] == bench.sources_hash(row)
    assert bench.recorded_traffic(row, bench.units_per_launch(row)) is not None
