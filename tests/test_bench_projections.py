"""bench.py --projections: the step from the residual stream back onto it, with and without
the norm + RoPE producer between the projections and the routing."""
import os
import subprocess
import sys

import pytest

from test_bench_contract import ROOT, _check_base, _run


@pytest.mark.gpu
@pytest.mark.parametrize("more", [[], ["--producer"]])
def test_line_with_projections(more):
    d = _run(["--config", "tiny", "--steps", "3", "--warmup", "3", "--projections", "--no-cpu-baseline", *more], 900)
    _check_base(d)
    assert d["config"]["projections"] and "e2e" not in d
    plain = _run(["--config", "tiny", "--steps", "3", "--warmup", "3", "--no-cpu-baseline", "--no-e2e", "--no-parity",
                  *more], 900)
    assert d["gpu_launches"] == plain["gpu_launches"] + 7 * 3
    p = d["parity"]
    assert p["ok"] is True and p["mask_mismatch"] == 0 and p["out_rows"] > 0


def test_pruning_is_refused():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--projections", "--prune", "0.5"], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 2 and "choose one" in out.stderr
