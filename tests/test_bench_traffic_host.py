"""bench.py reports each workload's DRAM traffic from a capture of the kernel sources
as they are: when one of them changes, the capture is taken again and its hash noted
beside the figure, so that no line loses it."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


@pytest.mark.parametrize("workload", bench.WORKLOADS)
def test_traffic_is_of_the_present_sources(workload):
    got, note = bench.traffic_of(workload)
    assert got is not None, note
    assert os.path.exists(os.path.join(ROOT, note))
