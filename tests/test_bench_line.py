"""What bench.py prints and reads, without a GPU."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_profiled_traffic_belongs_to_the_present_sources():
    """A summary's DRAM traffic is reported only while the sources it names are unchanged: a
    change to them wants a new capture."""
    for kernel in bench.KERNEL_SOURCES:
        assert bench.profiled_traffic(kernel, "4096x4096x2048_v64m8") is not None, kernel
