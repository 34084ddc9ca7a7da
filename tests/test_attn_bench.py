"""bench.py --attention: off by default, and only for the layer workloads."""
import sys

import pytest

import bench


def test_attention_flag_goes_with_layer_workloads(monkeypatch):
    monkeypatch.setattr(sys, "argv", ["bench.py", "--attention"])
    a = bench.parse()
    assert a.attention and a.workload == "llama2_7b_prefill" and a.context == 2048
    monkeypatch.setattr(sys, "argv", ["bench.py"])
    assert not bench.parse().attention
    for bad in (["--attention", "--workload", "mlp_block"], ["--attention", "--workload", "l2qer_compare"],
                ["--attention", "--context", "-1"]):
        monkeypatch.setattr(sys, "argv", ["bench.py"] + bad)
        with pytest.raises(SystemExit):
            bench.parse()
