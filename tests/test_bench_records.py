"""The committed traffic records are those of the GEMM as it stands, so that
the benchmark reports them."""
import glob
import os

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORDS = sorted(glob.glob(os.path.join(ROOT, "profiles", "gemm_traffic_*.txt")))


@pytest.mark.parametrize("path", RECORDS, ids=os.path.basename)
def test_records_are_of_the_present_sources(path):
    workload = os.path.basename(path)[len("gemm_traffic_"):-len(".txt")]
    traffic, how = bench.recorded_traffic(workload)
    assert traffic is not None and traffic > 0, how


def test_headers_of_the_gemm_hold_nothing_of_the_operators():
    for name in ("ptx.cuh", "kernels.h"):
        with open(os.path.join(ROOT, "w8a8_int8_linear_gb300", "csrc", name)) as f:
            text = f.read().lower()
        for word in ("attention", "rotary", "residual"):
            assert word not in text, (name, word)
