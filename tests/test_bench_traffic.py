"""The measured DRAM traffic that bench.py reports belongs to the kernels' sources as they are."""
import sys

import pytest

import synth
from conftest import ROOT

sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("config,path,fingerprint", sorted(bench.NCU_TRAFFIC))
def test_traffic_is_of_these_sources(config, path, fingerprint):
    family = path if path in ("compress", "split") else bench.kernel_family(synth.WORKLOADS[config], path)
    assert bench.kernel_fingerprint(family) == fingerprint
