"""The benchmark's measured traffic: every workload that has a capture reports it."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


@pytest.mark.parametrize("name", ["c2", "c3", "c4", "c5"])
def test_captures_are_of_the_present_sources(name):
    """The GEMM sources are those that the captures were taken on, so that the roofline has a
    traffic.  (An edit of their code wants new captures of these workloads.)"""
    import bench
    import synth
    cfg = synth.get_config(name)
    assert cfg.name in bench.TRAFFIC_PROFILES
    traffic = bench.gemm_traffic(cfg)
    assert traffic is not None and traffic > 1e8
