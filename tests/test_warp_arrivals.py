"""A warp whose lane 0 arrives at a barrier for all of its lanes (they have read
a buffer that asynchronous copies overwrite next, or written one) has met before:
nothing else orders the other lanes' accesses before the arrival.  No run shows
a missing meeting as long as the compiler keeps the warp together, so this looks
at the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "dsa_sparse_attention_index_gb300", "csrc")
MEETINGS = re.compile(r"__syncwarp\(|__syncthreads|bar_\w+\(")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_lanes_meet_before_lane_0_arrives_for_them(path):
    lines = open(path).read().split("\n")
    for i, line in enumerate(lines):
        if re.search(r"lane == 0\) mbar_arrive\(", line):
            # back to the last meeting, over nothing but statements that touch no memory
            before = i - 1
            while re.fullmatch(r"\s*(if \([a-z ]+\) \{|tc_fence_before\(\);|const bool last = .*)?(//.*)?", lines[before]):
                before -= 1
            assert MEETINGS.search(lines[before]), f"{os.path.basename(path)}:{i + 1}: {line.strip()}"
