"""The recorded DRAM traffic of the score kernel is valid for the kernel source
it was captured with: a change to that file asks for another capture."""
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_record_belongs_to_the_source():
    src = os.path.join(ROOT, "eviction_kvc_score_gb300", "csrc", "score_tc.cu")
    assert bench.traffic_for(src, "llama3_8b_zigzag_32L_T32768") is not None
    assert bench.traffic_for(src, "another workload") is None
