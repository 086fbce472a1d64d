"""Sums of the 8-bit floating-point products in every kernel: 32 bits, whatever y's
type.  Operands whose products cancel exactly beside small ones: a sum that keeps
fewer bits anywhere loses the small ones."""
import numpy as np
import pytest

from tests import epi_ref as R
from tests import fp8_ref as F
from tests.fp8_kernel import kernel

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a4_rank_corrected_amd as S
    S.lib()
    return S


def bf16(v):
    return torch.from_numpy(R.bf16_bits(v).view(np.int16)).cuda().view(torch.bfloat16)


def cancelling(rng, b, m, n, E=1):
    """(x [b][m], w [E][n][m], what x w^T is per expert): of every eight neighbouring channels two have products of
    448 x 448 and its opposite, one a product of 1, 2 or -1, the others none.  All are values of codes with the scale
    2^0 (every block's largest magnitude is 448); all sums of products are whole numbers below 2^24, which fp32 holds
    whatever their order, and each result is one of at most 256 in magnitude, which bf16 holds."""
    assert m % 128 == 0 and m // 8 <= 83  # 83 x 448 x 448 < 2^24
    x, w = np.zeros((b, m)), np.zeros((E, n, m))
    x[:, 0::8] = x[:, 1::8] = 448
    w[..., 0::8], w[..., 1::8] = 448, -448
    x[:, 2::8] = rng.choice([1.0, -1.0], (b, 1))
    at = rng.integers(0, 8, (E, n, m // 8))  # one group in eight has a part
    w[..., 2::8] = np.where(at == 0, rng.choice([1.0, 2.0], (E, n, m // 8)), 0.0)
    v = np.einsum("bk,enk->ebn", x[:, 2::8], w[..., 2::8])
    assert np.abs(v).max() <= 256
    return x, w, v


# one row and some, the row kernel in its three forms, tiles of 64 x 128, of 128 x 128, those in pieces; few rows of wide
# layers; and shapes of more than 128 tiles of 256 x 256
SHAPES = [(1, 128, 50), (16, 640, 300), (40, 256, 500), (150, 640, 1000), (700, 384, 1500), (2100, 640, 900), (300, 640, 700),
          (1, 128, 33024), (1, 640, 32768), (33, 640, 12288), (2300, 384, 4100), (4096, 128, 4096), (4350, 256, 4150)]


@pytest.mark.parametrize("b,m,n", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_sums_hold_32_bits(S, b, m, n, out):
    print(f"fp8 sums b={b} m={m} n={n} {out}: {kernel(b, n, m, 0, out)}", flush=True)
    x, w, v = cancelling(np.random.default_rng([b, m, n]), b, m, n)
    lay = S.DeviceLayerFp8(bf16(w[0]), transposed=True)
    y = S.svdq_fp8_linear(bf16(x), lay, out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    assert np.array_equal(y.float().cpu().numpy(), v[0])


GROUPED = [(8, 12, 256, 70), (4, 600, 256, 300), (64, 2500, 256, 1408), (8, 3000, 256, 700), (2, 2300, 256, 300)]


@pytest.mark.parametrize("E,b,m,n", GROUPED)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_sums_hold_32_bits_grouped(S, E, b, m, n, out):
    print(f"fp8 sums E={E} b={b} m={m} n={n} {out}: {kernel(b, n, m, E, out)}", flush=True)
    rng = np.random.default_rng([E, b, m, n])
    x, w, v = cancelling(rng, b, m, n, E)
    lay = S.GroupedDeviceLayerFp8(bf16(w), transposed=True)
    off = np.concatenate([[0], np.sort(rng.integers(0, b + 1, E - 1)), [b]])
    y = S.svdq_fp8_grouped_linear(bf16(x), torch.tensor(off, dtype=torch.int32).cuda(), lay,
                                  out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    want = np.concatenate([v[e, off[e]: off[e + 1]] for e in range(E)])
    assert np.array_equal(y.float().cpu().numpy(), want)


# ---------------------------------------------------------------------------
# the 8-bit matrix instruction, where a caller asks for it
# ---------------------------------------------------------------------------

FAST = [(700, 384, 1500, "small"), (2100, 640, 900, "tiles"), (300, 4608, 700, "pieces"), (2500, 1100, 300, "small"),
        (4350, 260, 4150, "big 4"), (2048, 1152, 4608, "big 1"), (4100, 140, 2300, "big 1"), (4096, 260, 4608, "big 4"),
        (4608, 130, 5376, "big 2")]


def values(rng, b, m, n, E=1):
    x = rng.standard_normal((b, m)) * np.exp(0.7 * rng.standard_normal((b, 1)))
    x[:, rng.choice(m, max(1, m // 60), replace=False)] *= 30
    w = rng.standard_normal((E, n, m)) / np.sqrt(m) * np.exp(0.4 * rng.standard_normal((E, n, 1)))
    return R.bf16(x), R.bf16(w)


@pytest.mark.parametrize("b,m,n,which", FAST)
def test_fast_sums(S, b, m, n, which):
    """Within the instruction's own bound; exact results of the same operands within theirs."""
    assert kernel(b, n, m, 0, "fast") == which
    rng = np.random.default_rng([b, m, n])
    x, w = values(rng, b, m, n)
    rows = np.unique(np.concatenate([[0, b - 1], rng.integers(0, b, 60)]))
    lay = S.DeviceLayerFp8(bf16(w[0]), transposed=True)
    xq, wq = F.quantize(x[rows], 1), F.quantize(w[0], 128)
    v, dv = R.product_values(xq[2], wq[2], m)
    for fast in (True, False):
        y, bound = R.epilogue(v, dv + (F.aligned(xq, wq) if fast else 0), "silu", out="bf16")
        got = S.svdq_fp8_linear(bf16(x), lay, act="silu", out_dtype=torch.bfloat16, fast_sums=fast).float().cpu().numpy()[rows]
        assert (np.abs(got - y) <= bound).all(), fast


@pytest.mark.parametrize("E,b,m,n,which", [(8, 3000, 260, 700, "tiles"), (2, 2300, 260, 300, "big 1"), (8, 12, 256, 70, "rows 1")])
def test_fast_sums_grouped(S, E, b, m, n, which):
    assert kernel(b, n, m, E, "fast") == which
    rng = np.random.default_rng([E, b, m, n])
    x, w = values(rng, b, m, n, E)
    off = np.concatenate([[0], np.sort(rng.integers(0, b + 1, E - 1)), [b]])
    od = torch.tensor(off, dtype=torch.int32).cuda()
    lay = S.GroupedDeviceLayerFp8(bf16(w), transposed=True)
    got = S.svdq_fp8_grouped_linear(bf16(x), od, lay, fast_sums=True)
    qx, asc = S.svdq_fp8_quantize_act(bf16(x))
    assert torch.equal(S.svdq_fp8_grouped_gemm(qx, asc, od, lay, fast_sums=True), got)
    got = got.float().cpu().numpy()
    for e in range(E):
        s = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        xq, wq = F.quantize(x[s], 1), F.quantize(w[e], 128)
        v, dv = R.product_values(xq[2], wq[2], m)
        y, bound = R.epilogue(v, dv + F.aligned(xq, wq), out="bf16")
        assert (np.abs(got[s] - y) <= bound).all(), e


def test_fast_sums_take_bf16_only(S):
    x, w = values(np.random.default_rng(0), 4, 200, 30)
    lay = S.DeviceLayerFp8(bf16(w[0]), transposed=True)
    qx, asc = S.svdq_fp8_quantize_act(bf16(x))
    for call in (lambda d: S.svdq_fp8_linear(bf16(x), lay, out_dtype=d, fast_sums=True),
                 lambda d: S.svdq_fp8_gemm(qx, asc, lay, out_dtype=d, fast_sums=True)):
        with pytest.raises(ValueError, match="bfloat16"):
            call(torch.float32)
        # few rows are added exactly either way
        assert torch.equal(call(torch.bfloat16), S.svdq_fp8_linear(bf16(x), lay, out_dtype=torch.bfloat16))
