"""The bench's DRAM traffic of a kernel is that of the sources it was captured on (CPU only)."""
import json

import pytest

import bench
from dynamic_sparse_attention_estimate_gb300.inputs import WORKLOADS

STORED = json.load(open(bench.TRAFFIC_FILE))


@pytest.mark.parametrize("kernel", sorted(STORED))
def test_stored_traffic_belongs_to_the_current_sources(kernel):
    """One that does not is left out of the bench's line: captured anew, or taken out of the file, when a kernel changes."""
    assert STORED[kernel]["source_hash"] == bench.kernel_source_hash(kernel)


def test_the_long_clip_reports_its_traffic():
    prof = {"bwd_main": (120, 1200.0), "bwd_reduce": (120, 400.0), "sparse_fwd": (6, 690.0)}
    assert bench.roofline(prof, 1, WORKLOADS["long"])["traffic"] > 0
