"""CPU tests of the rows' gradient: its workgroups cover the rows, and what the C ABI
does without any row or token."""
import ctypes
import os
import subprocess

import pytest

pytest.importorskip("w4a4_rank_corrected_amd")
from w4a4_rank_corrected_amd import _binding as B  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_rank_corrected_amd", "csrc")


def test_plan_covers_the_rows(tmp_path):
    src = tmp_path / "q.cpp"
    src.write_text('#include "internal.h"\nextern "C" void q(int R, int* out) {\n'
                   "  const svdq::GradPlan p = svdq::grad_plan(R);\n  out[0] = p.per;\n  out[1] = p.blocks;\n}\n")
    so = str(tmp_path / "q.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", str(src),
                    os.path.join(CSRC, "plan.cpp"), "-o", so], check=True, capture_output=True)
    q = ctypes.CDLL(so).q
    v = (ctypes.c_int * 2)()
    for R in (1, 2, 511, 512, 513, 1025, 24576, 100003, 1 << 20, 2097152, 2097153, B.SVDQ_MAX_DIM - 1, B.SVDQ_MAX_DIM):
        q(R, v)
        per, blocks = v
        assert 1 <= per <= 4096 and blocks * per >= R > (blocks - 1) * per, (R, per, blocks)


def test_nothing_to_do():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libsvdq.so not built")
    L = B.lib()
    f = 0x10000
    assert L.svdq_combine_rows_grad(None, 0, 8, 0, None, None, 2, f, 5, f << 2, f << 4, None) == B.SVDQ_OK
    assert L.svdq_combine_rows_grad(f, 4, 8, 0, f << 1, None, 2, None, 0, f << 2, None, None) == B.SVDQ_OK
    assert L.svdq_combine_rows_grad(f, 4, 8, 0, f << 1, None, 2, f << 3, 5, None, None, None) == B.SVDQ_OK
