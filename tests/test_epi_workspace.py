"""Host code of the products with an epilogue and of the grouped layers, built
with stubs for the launchers: the workspaces that calls ask for
(tests/native/epi_workspace.cpp) and the largest grouped products
(tests/native/grouped_limits.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_rank_corrected_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")


@pytest.mark.parametrize("program,says", [("epi_workspace", "epi workspace ok"), ("grouped_limits", "grouped limits ok")])
def test_host_checks(tmp_path, program, says):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / program)
    sources = [os.path.join(CSRC, f) for f in ("api.cpp", "epi_api.cpp", "prep.cpp", "bundle.cpp", "plan.cpp")] + \
              [os.path.join(NATIVE, f) for f in ("device_stubs.cpp", "epi_stubs.cpp", program + ".cpp")]
    res = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                          "-fno-sanitize-recover=undefined", "-ffp-contract=off", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
                          *sources, "-o", exe, "-pthread"], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and says in run.stdout, (run.stdout + run.stderr)[-4000:]
