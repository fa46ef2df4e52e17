"""The committed summaries of HBM traffic belong to the library's sources: a
bench line gives a sweep's traffic from them, and none from a summary taken on
other sources (those that define the sweeps' code and launches)."""
import glob
import json
import os

import pytest

from rl_policy_gradient_amd import profsum

FILES = sorted(glob.glob(os.path.join(profsum.ROOT, "profiles", "traffic_*.json")))


def test_there_are_summaries():
    assert any("wgrad_sweep_gmpo_bf16_b128_t32768_chunked" in f for f in FILES)  # the default line's


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_taken_on_these_sources(path):
    import bench
    with open(path) as fh:
        d = json.load(fh)
    assert d["kernel_src_hash"] == profsum.kernel_src_hash(), "take it again: profsum's `traffic`, by its `command`"
    assert bench._traffic_from_profiles(d["kernel"], d["workload"]) == d["bytes_per_launch"] > 0
