"""The gradients of combine and dispatch in the bounds-checked build (-DMOE_BOUNDS_CHECK: a row that the map or the
search gives is checked against the receive buffers; a miss records MOE_ERR_OUT_OF_BOUNDS): same results, status OK. In a
child process, as the library is loaded once per process (CRS_MOE_CHECKED=1 picks the checked one)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SELECTION = {
    "tests/test_gradients_gpu.py": "test_combine_backward or test_dispatch_backward or another_order or do_not_match or "
                                   "two_batches or training_step",
    "tests/test_gradients_map_gpu.py": "rebuilt or another_order or do_not_match or replayed",
}


@pytest.mark.parametrize("path", SELECTION)
def test_checked_build_runs_the_gradients(path):
    from combine_route_scan_gb300 import build as B
    lib = B.build(checked=True)
    assert os.path.exists(lib)
    env = {k: v for k, v in os.environ.items() if k not in ("CRS_MOE_CHECKED", "CRS_MOE_OBSERVER", "CRS_MOE_PHASE")}
    env["CRS_MOE_CHECKED"] = "1"
    probe = subprocess.run([sys.executable, "-c", "from combine_route_scan_gb300 import moe; print(moe.lib()._name)"],
                           cwd=ROOT, env=env, capture_output=True, text=True, timeout=120)
    assert probe.returncode == 0 and os.path.join("_build", "checked") in probe.stdout, probe.stdout + probe.stderr
    r = subprocess.run([sys.executable, "-m", "pytest", path, "-k", SELECTION[path], "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, f"{r.stdout[-3000:]}\n{r.stderr[-2000:]}"
    assert " passed" in r.stdout and "failed" not in r.stdout
