"""The committed DRAM-traffic records belong to the committed kernels: bench.py
reports no traffic for a kernel whose source has changed since its record."""
import json
import os

import pytest

import bench

PREFILL = ["gemm_tc.cuh", "common.cuh"]
DECODE = ["gemv_stream.cuh", "gemv_decode.cuh", "common.cuh"]
RECORDS = {"llama2_7b_prefill": PREFILL, "llama2_7b_decode_M16": DECODE, "mlp_block": PREFILL, "llama3_8b_w4a8": PREFILL}


@pytest.mark.parametrize("name", sorted(RECORDS))
def test_record_is_of_the_committed_kernel(name):
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        rec = json.load(f)
    assert sorted(rec) == sorted(RECORDS)
    assert bench.recorded_traffic(name, RECORDS[name]) == rec[name]["bytes_per_launch"]
