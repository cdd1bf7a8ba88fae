"""The benchmark's DRAM-traffic figures are stored captures of the layer's GEMM kernels, valid while those kernels'
sources are what was captured: what other operators need goes into files of their own."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("workload,stage", list(bench.MEASURED_TRAFFIC))
def test_the_captures_are_of_these_sources(workload, stage):
    nbytes, where = bench.measured_traffic(workload, stage)
    assert nbytes == bench.MEASURED_TRAFFIC[workload, stage][0], where
