"""The counter profiles that bench.py reports beside its times belong to the GEMM kernels of this tree (CPU)."""
import glob
import json
import os

import pytest

import bench

PROFILES = sorted(glob.glob(os.path.join(bench.ROOT, "profiles", "traffic_*.json")))


def test_there_are_profiles():
    assert len(PROFILES) >= 5


@pytest.mark.parametrize("path", PROFILES, ids=lambda p: os.path.basename(p)[8:-5])
def test_profile_is_reported(path):
    traffic, note = bench.load_traffic(os.path.basename(path)[8:-5], bench.kernel_source_sha())
    assert traffic is not None, note
    assert json.load(open(path))["kernel_src_sha"] == bench.kernel_source_sha()
