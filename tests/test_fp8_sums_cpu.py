"""CPU tests of the choice of sums in the 8-bit floating-point products: what takes
the flag, and the workspace for either choice."""
import ctypes
import os

import pytest

from tests.fp8_kernel import kernel, workspace

pytest.importorskip("w4a4_rank_corrected_amd")
from w4a4_rank_corrected_amd import _binding as B  # noqa: E402

FAKE = 0x10000  # never dereferenced: every call below is refused
FAST = B.SVDQ_FP8_FAST_SUMS
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libsvdq.so not built")
    return B.lib()


def test_flag_is_for_bf16_results_of_this_setting(L):
    lay = ctypes.byref(B.svdq_fp8_layer(200, 64, FAKE, FAKE, None))
    group = ctypes.byref(B.svdq_fp8_grouped_layer(4, 200, 64, FAKE, FAKE, None))
    for t in (B.SVDQ_OUT_F32 | FAST, 2 | FAST, FAST << 1, 2):
        for status in (L.svdq_fp8_gemm(FAKE, FAKE, lay, None, 16, FAKE, t, FAKE, BIG, None),
                       L.svdq_fp8_linear(FAKE, lay, None, 16, FAKE, t, FAKE, BIG, None),
                       L.svdq_fp8_grouped_gemm(FAKE, FAKE, 16, None, FAKE, group, None, 16, FAKE, t, None),
                       L.svdq_fp8_grouped_linear(FAKE, 16, None, FAKE, group, None, 16, FAKE, t, FAKE, BIG, None)):
            assert status == B.SVDQ_ERR_INVALID_ARG, t
    # with the flag the other checks are the same: a missing workspace, a misaligned y, no rows
    t = B.SVDQ_OUT_BF16 | FAST
    assert L.svdq_fp8_linear(FAKE, lay, None, 16, FAKE, t, None, 0, None) == B.SVDQ_ERR_WORKSPACE
    assert L.svdq_fp8_linear(FAKE, lay, None, 16, FAKE + 1, t, FAKE, BIG, None) == B.SVDQ_ERR_ALIGNMENT
    assert L.svdq_fp8_linear(None, lay, None, 0, None, t, None, 0, None) == B.SVDQ_OK
    layer4 = ctypes.byref(B.svdq_layer(m=64, n=64, rank=0, group=64, qw=FAKE, wscale=FAKE))
    assert L.svdq_linear_epi(FAKE, layer4, None, 16, FAKE, t, FAKE, BIG, None) == B.SVDQ_ERR_INVALID_ARG
    assert b"y_dtype" in L.svdq_last_error()


SIZES = (1, 16, 17, 64, 65, 128, 300, 333, 512, 1000, 2048, 4096, 4608, 12288, 270000)


def test_workspace_serves_either_choice(L):
    for b in SIZES:
        for n in SIZES:
            for m in (1, 128, 640, 1152, 2048, 4608, 16384):
                need = L.svdq_fp8_gemm_workspace_size(b, n, m)
                assert need >= max(workspace(b, n, m, out) for out in ("bf16", "f32", "fast")), (b, n, m)


def test_exact_sums_unless_asked_for():
    """Tiles of 256 x 256 are the 8-bit instruction's; few rows take the row kernel or exact tiles of any kind."""
    for b in SIZES:
        for n in SIZES:
            for m in (128, 1152, 4608):
                for E in (0, 8):
                    assert not kernel(b, n, m, E, "bf16").startswith("big"), (b, n, m, E)
                    assert kernel(b, n, m, E, "bf16") == kernel(b, n, m, E, "f32")


# weights of some MB to 500 MB: up-projections, output layers
WIDE = [(1152, 6912), (1152, 32768), (128, 33024), (4096, 14336), (4096, 32769), (4096, 128256), (8192, 8192), (8192, 28672),
        (16384, 7168), (2048, 32000), (2048, 65536), (8192, 65536)]


@pytest.mark.parametrize("m,n", WIDE)
@pytest.mark.parametrize("out", ["bf16", "f32", "fast"])
def test_one_row_of_a_wide_layer_takes_the_row_kernel(m, n, out):
    """It reads the weights at memory's rate; tiles of 64 rows and more leave all but one of them empty."""
    assert kernel(1, n, m, 0, out) == "rows 1"


@pytest.mark.parametrize("m,n", WIDE)
def test_few_rows_take_no_tiles_of_256_rows(m, n):
    for b in (1, 16, 64, 128):
        assert not kernel(b, n, m, 0, "fast").startswith("big")
