"""Which kernel a product in 8-bit floating point takes: the library's own plan
(csrc/plan.cpp), built for the host."""
import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_rank_corrected_amd", "csrc")


@functools.lru_cache(maxsize=None)
def _query():
    at = tempfile.mkdtemp(prefix="fp8_plan_")
    so = os.path.join(at, "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-ffp-contract=off", f"-I{os.path.join(ROOT, 'include')}",
                    f"-I{CSRC}", os.path.join(CSRC, "plan.cpp"), os.path.join(ROOT, "tests", "native", "fp8_plan_query.cpp"),
                    "-o", so], check=True, capture_output=True, text=True)
    return ctypes.CDLL(so).fp8_plan_query


def _plan(b, n, m, experts, out):
    v = (ctypes.c_int * 6)()
    _query()(b, n, m, experts, {"bf16": 0, "f32": 1, "fast": 0x100}[out], v)
    return list(v)


def workspace(b, n, m, out):
    """Bytes that the product's kernels write."""
    return _plan(b, n, m, 0, out)[5] << 16


def kernel(b, n, m, experts=0, out="bf16"):
    """out: 'bf16', 'f32' or 'fast' (bf16 with the sums of the 8-bit matrix instruction).  'rows 1' / 'rows 2' / 'rows 4' (16-row blocks of the row kernel), 'small' (tiles of 64 x 128), 'tiles' (128 x
    128), 'pieces' (those split along the channels), 'big 1' / 'big 2' / 'big 4' (256 x 256, parts of the last round)."""
    rb, big, small, parts, pieces, _ = _plan(b, n, m, experts, out)
    if rb:
        return f"rows {rb}"
    if big:
        return f"big {parts}"
    return "small" if small else ("pieces" if pieces > 1 else "tiles")
