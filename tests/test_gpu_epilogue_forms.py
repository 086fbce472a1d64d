"""Products with an epilogue, the forms that differ between the settings and
between their kernels: the 8-bit product on both sides of the choice between
small tiles and pieces."""
import pytest

from tests.test_gpu_epilogue import Case, S, _say  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# 64 x 64 tiles: up to about 40 groups of few tiles, one round or less of 64 x 64 tiles, 512 of them; pieces: 49 to 128
# groups of few tiles, a little past a round; the plain plan (390 wide tiles)
@pytest.mark.parametrize("rank", [0, 24])
@pytest.mark.parametrize("b,m,n", [(1, 2048, 130), (256, 2048, 1152), (400, 4032, 1152), (1000, 4096, 2048),
                                   (1, 3136, 70), (100, 4032, 500), (256, 4032, 1152), (65, 8192, 333), (600, 5120, 2048),
                                   (1600, 512, 3840)])
def test_8bit_small_tiles_and_pieces(S, b, m, n, rank):
    _say(f"w8a8 b={b} m={m} n={n} rank={rank}")
    c = Case(S, "w8a8", b, m, n, rank, bias=rank == 0)
    c.run(act="gelu_erf", act_begin=n // 3, gate_rows=max(1, b // 3), residual=True, out="bf16", inplace=True)
    c.run(out="f32")
