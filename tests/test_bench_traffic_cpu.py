"""The bench reports the forward kernel's measured DRAM traffic only while the kernel's
sources are those of the capture; a helper that another kernel needs belongs elsewhere."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_the_traffic_figure_belongs_to_the_sources_in_the_tree():
    assert (bench.sources_digest(bench.ATTEND_FWD_SOURCES)
            == bench.ATTEND_FWD_TRAFFIC["sources_sha256"])
    assert bench.ATTEND_FWD_TRAFFIC["bytes"] > 0
