"""bench.py's traffic field comes from the committed counter summaries, which count as long as the
scan's sources are those that they were taken of."""
import os

import pytest

import bench


@pytest.mark.parametrize("name", [f[len("scan_forward_"):-len(".md")] for f in sorted(os.listdir(bench.COUNTERS_DIR))
                                  if f.startswith("scan_forward_") and "wavefront" not in f])
def test_the_summary_is_of_these_sources(name):
    assert bench.recorded_traffic(name) is not None, (
        "profiles/scan_forward_%s.md is of other sources (now %s): take it again" % (name, bench.scan_source_hash()))
