"""The DRAM traffic that the benchmark reports with its roofline belongs to the kernels as they are."""
import pytest

import bench


@pytest.mark.parametrize("key", sorted(bench.NCU_TRAFFIC))
def test_recorded_traffic_is_of_the_present_source(key):
    nbytes, note = bench.traffic_for(*key)
    assert nbytes == bench.NCU_TRAFFIC[key]["bytes"], note
