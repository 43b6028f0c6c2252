"""What bench.py prints and reads, without a GPU."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_profiled_traffic_belongs_to_the_present_sources():
    """A summary's DRAM traffic is reported only while the sources it names are unchanged: a
    change to them wants a new capture."""
    for kernel in bench.KERNEL_SOURCES:
        assert bench.profiled_traffic(kernel, "4096x4096x2048_v64m8") is not None, kernel


def test_one_short_line_with_the_contract_keys(capsys):
    """The table of workloads, most of the output, goes to stderr; every other key is on stdout."""
    text = "x" * 250
    nested = {f"part_{i}_per_step": 0.12345678901234567 * 10 ** i for i in range(8)}
    line = {"metric": bench.METRIC, "value": 1146.761925213188, "unit": "TFLOP/s", "n_gpus": 1, "steps": 20, "warmup": 5,
            "ms_per_step": 0.05992479801177979, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
            "dtype": "f16", "data": "synthetic", "config": {"workload": text}, "step_schedule": {**nested, "pipelined": text},
            "kernels": nested, "roofline": {**nested, "per_launch": text}, "cpu_baseline": {**nested, "sample": text},
            "e2e": {"value": 253.8336789214771, "h2d_bytes_per_step": 50331648, "d2h_bytes_per_step": 16777216},
            "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": []}, "gpu_launches": 600,
            "per_config": {"cases": [nested] * 100}}
    bench.print_line(line)
    out, err = capsys.readouterr()
    assert out.count("\n") == 1 and len(out) < 3000
    got = json.loads(out)
    assert set(got) == set(line) - {"per_config"}
    assert abs(got["value"] / line["value"] - 1) < 1e-6 and got["e2e"]["h2d_bytes_per_step"] == 50331648
    assert json.loads(err)["per_config"] == line["per_config"] and "per_config" in line
