"""What the bench and the build say about the sources they were made with."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def test_profiled_traffic_is_of_the_present_forward_kernel():
    import bench
    for name, rec in bench.PROFILED_TRAFFIC.items():
        assert bench.kernel_traffic(name) == rec["bytes"]
