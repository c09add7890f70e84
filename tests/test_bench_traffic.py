"""The DRAM traffic that the benchmark reports beside its dominant kernel comes from a
committed capture, and only while the kernel's sources are those of the capture."""

import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("kernel", ["attn_bwd_causal", "attn_fwd"])
def test_the_capture_is_of_the_committed_sources(kernel):
    spec = importlib.util.spec_from_file_location("bench_module", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    assert bench.traffic_for(kernel, "long_ttt") is not None
