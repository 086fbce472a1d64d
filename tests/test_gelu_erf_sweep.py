"""Host sweep of the GELU_ERF evaluation (tests/native/gelu_erf_sweep.c), with the
constants that csrc/epilogue.h holds: Phi stays within the 1e-7 that the header
promises, for any 2^x within an ulp.  A planted mistake (a constant off in its
fifth digit) must be caught."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "native", "gelu_erf_sweep.c")
ROOT = os.path.dirname(HERE)


def _promised():
    text = open(os.path.join(ROOT, "include", "svdq.h")).read()
    return float(re.search(r"GELU_ERF\s+v Phi\(v\) \(Phi to an absolute error of at most (\S+);", text).group(1))


def _constants():
    text = open(os.path.join(ROOT, "w4a4_rank_corrected_amd", "csrc", "epilogue.h")).read()
    body = re.search(r"kPhi\[10\] = \{([^}]*)\}", text).group(1)
    return [c.strip().rstrip("f") for c in body.split(",")]


@pytest.fixture(scope="module")
def sweep(tmp_path_factory):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    exe = str(tmp_path_factory.mktemp("ge") / "sweep")
    with open("/proc/cpuinfo") as f:
        fma = ["-mfma"] if " fma " in f.read() else []
    subprocess.check_call(["gcc", "-O2", "-fopenmp", "-ffp-contract=off", "-fno-fast-math", *fma, "-o", exe, SRC, "-lm"])

    def run(constants, step):
        out = subprocess.run([exe, str(step), *constants], capture_output=True, text=True, timeout=600, check=True).stdout
        count, worst, at = out.split()
        return int(count), float(worst), float(at)

    return run


def test_phi_stays_within_the_promise(sweep):
    count, worst, at = sweep(_constants(), 1)
    assert count == 0x7F800000 - 0x30000000
    assert _promised() == 1e-7
    assert worst <= _promised(), (worst, at)


def test_a_wrong_constant_is_caught(sweep):
    c = _constants()
    c[1] = repr(float(c[1]) * (1 + 1e-5))
    assert not sweep(c, 61)[1] <= _promised()
