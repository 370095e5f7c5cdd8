"""The DRAM traffic that bench.py takes from the committed profiles."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("kernel,workload", [("opd_fast_kernel", "mix:verify_T1+opd"), ("verify_stats", "mix:verify_T0.6")])
def test_traffic_is_of_the_current_sources(kernel, workload):
    """A change of a kernel's sources calls for a new capture; a change of other
    kernels' does not touch them."""
    import bench
    assert bench._profile_traffic(kernel, workload) is not None
