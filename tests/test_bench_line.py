"""What bench.py prints: one short JSON line on stdout with the headline, all
figures of parts and other configurations on stderr."""
import json

import bench

LINE = {
    "metric": bench.METRIC, "value": 1.0 / 3, "unit": "tokens/s", "n_gpus": 1, "steps": 20, "warmup": 5,
    "ms_per_step": 1.0 / 3, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
    "data": "synthetic", "config": {"workload": "long_seq_train", "l2": "inputs larger than L2 (no flush)"},
    "roofline": {"achieved": 1.0 / 3}, "block_roofline": {"frac": 1.0 / 3}, "cpu_baseline": {"value": 1.0},
    "e2e": {"value": 1.0 / 3, "unit": "tokens/s", "h2d_bytes_per_step": 1, "d2h_bytes_per_step": 1},
    "gpu_launches": 180, "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": []},
    "kernels": {f"kernel{i}": {"median_us": i / 3, "frac": i / 7} for i in range(11)},
    "fwd_tokens_per_s": 2.0 / 3, "mxfp8_forward": {"value": 1.0}, "mxfp8_train": {"value": 1.0},
    "configs": [{"workload": f"w{i}", "kernels": {f"kernel{j}": j / 3 for j in range(40)}} for i in range(20)],
}


def test_one_short_line_and_the_details_apart(capsys):
    bench.emit(LINE)
    out, err = capsys.readouterr()
    lines = out.splitlines()
    assert len(lines) == 1 and len(lines[0]) < 4000
    headline = json.loads(lines[0])
    assert set(LINE) - set(headline) == {"kernels", "mxfp8_forward", "mxfp8_train", "configs"}
    assert all(headline[k] == LINE[k] for k in headline)
    assert json.loads(err) == LINE
