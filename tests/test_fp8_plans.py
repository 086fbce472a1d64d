"""The host code of the 8-bit floating-point setting and of the routing, built with
stubs for the launchers and run under the sanitizers (tests/native/fp8_plans.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_rank_corrected_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")


def test_plans_and_workspaces(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "fp8_plans")
    sources = [os.path.join(CSRC, f) for f in ("api.cpp", "epi_api.cpp", "fp8_api.cpp", "route_api.cpp", "prep.cpp", "bundle.cpp",
                                               "plan.cpp")] + \
              [os.path.join(NATIVE, f) for f in ("device_stubs.cpp", "epi_stubs.cpp", "fp8_stubs.cpp", "fp8_plans.cpp")]
    res = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                          "-ffp-contract=off", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", *sources, "-o", exe,
                          "-pthread"], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and "fp8 plans ok" in run.stdout, (run.stdout + run.stderr)[-4000:]
