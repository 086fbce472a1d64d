"""Exhaustive host proof of the grouped activation kernel's INT4 quantizer
(tests/native/quant_snap_exhaustive.c): its scales and codes equal the
definition's for every bf16 group maximum and value, for any reciprocal within
an ulp.  A planted mistake (a coarser snap) must be caught."""
import os
import shutil
import subprocess

import numpy as np
import pytest

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "quant_snap_exhaustive.c")


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    d = tmp_path_factory.mktemp("qs")
    exe, table = str(d / "check"), str(d / "table.bin")
    with open("/proc/cpuinfo") as f:
        fma = ["-mfma"] if " fma " in f.read() else []  # the same results, without a library call each
    subprocess.check_call(["gcc", "-O2", "-fopenmp", "-ffp-contract=off", "-fno-fast-math", *fma, "-o", exe, SRC, "-lm"])
    a = (np.arange(32768, dtype=np.uint32) << np.uint32(16)).view(np.float32)
    with np.errstate(all="ignore"):
        quo = np.where(np.isfinite(a), np.minimum(a / np.float32(7), np.float32(65504)), 0).astype(np.float32)
        tab = quo.astype(np.float16).view(np.uint16)
    with open(table, "wb") as f:
        f.write(tab.tobytes() + quo.tobytes())
    return exe, table


def test_scales_and_codes_match_the_definition(checker):
    res = subprocess.run([*checker], capture_output=True, text=True, timeout=600)
    scales, pairs, bad, ties = map(int, res.stdout.split())
    assert scales == 0x7F80 - 1 and pairs > 3e9 // 2 and ties > 0
    assert res.returncode == 0 and bad == 0


def test_a_coarser_snap_is_caught(checker):
    res = subprocess.run([*checker, "coarse"], capture_output=True, text=True, timeout=600)
    assert res.returncode == 1 and int(res.stdout.split()[2]) > 0
