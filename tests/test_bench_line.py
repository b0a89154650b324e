"""bench.py's own arm prints one short JSON line, whatever else it measured.  No GPU:
the measurement is replaced by its result."""
import json
import sys

import pytest
import torch

import bench
from synth import NANO_DECODE

KEYS = {"metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
        "vs_baseline", "dtype", "data", "config", "clocks", "e2e", "gpu_launches"}


@pytest.mark.parametrize("points", [0, 60])
def test_the_line_is_short_and_the_points_are_beside_it(monkeypatch, capsys, points):
    point = {f"figure_{i}": 0.123456789 for i in range(16)}
    result = dict(shape=NANO_DECODE, T=64, peaks=bench.peaks(), n_active=96, ms_per_step=0.38, value=166000.0, n_rep=2,
                  rep_bytes=2.6e9, routing={}, clocks={"sm_mhz": 2070}, launches=160, ms_eager=0.4, err=0, e2e_s=4e-4,
                  per_workload={f"workload T={i}": point for i in range(points)}, per_workload_clocks={})
    monkeypatch.setattr(bench, "run_ours", lambda *a: result)
    monkeypatch.setattr(bench, "roofline_entry", lambda *a: {})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(sys, "argv", ["bench.py", "--steps", "20", "--warmup", "5", "--no-cpu-baseline"])
    for name in ("WORLD_SIZE", "RANK", "LOCAL_RANK"):
        monkeypatch.delenv(name, raising=False)
    bench.main()
    out, err = capsys.readouterr()
    assert out.count("\n") == 1 and len(out) <= 4096
    line = json.loads(out)
    assert KEYS <= set(line) and line["value"] == 166000.0 and line["steps"] == 20
    if points:
        assert len(json.loads(err)["per_workload"]) == points
    else:
        assert err == ""
