"""The bench's DRAM traffic comes from committed captures that are taken for current
only while the kernels' sources are those that were captured."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


@pytest.mark.parametrize("kernel", ["scatter", "combine_reduce"])
def test_traffic_of_the_default_workload_is_current(kernel):
    """What other kernels need beside them stays out of the headers that these are built from."""
    import bench
    assert bench.committed_traffic(kernel, bench.DEFAULT_WORKLOAD) is not None
