"""The largest weights of the 8-bit floating-point setting: scales up to 2^120."""
import numpy as np
import pytest

from tests import epi_ref as R
from tests import fp8_ref as F
from tests.test_gpu_fp8 import S, close, dev_bf16  # noqa: F401 (S: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TOP = float(np.finfo(np.float32).max)


def large(rng, n, m, out):
    """[n][m]: blocks whose largest magnitudes lie from 2^120 to the type's largest value, all finite."""
    w = rng.standard_normal((n, m)) * 2.0 ** 120
    w[:128, :128] = rng.uniform(-0.99, 0.99, (128, 128)) * TOP
    w[5, 7] = TOP if out == "f32" else float.fromhex("0x1.fep127")  # the largest bf16 value
    w[128:, :128] *= 2.0 ** 4
    w[130, 5] = 1.75 * 2.0 ** 127  # the last one that the scale 2^119 brings to 448
    w[0, 130] = -1.75 * 2.0 ** 127 * (1 + 2.0 ** -7)
    w = R.bf16(w) if out == "bf16" else w.astype(np.float32).astype(np.float64)
    assert np.isfinite(w).all() and np.abs(w).max() <= TOP
    return w


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True])
def test_codes_of_the_largest_weights(S, out, transposed):  # noqa: F811
    n, m = 200, 300
    w = large(np.random.default_rng(1), n, m, out)
    wd = torch.from_numpy(np.ascontiguousarray(w if transposed else w.T)).to(torch.float32 if out == "f32" else torch.bfloat16).cuda()
    qw, ws = S.svdq_fp8_quantize_weights(wd, transposed=transposed)
    codes, es, _ = F.quantize(w, 128)
    assert es.max() == 120 and es[1, 0] == 119 and es[0, 1] == 120 and (codes != F.NAN).all()
    assert np.array_equal(qw.cpu().numpy(), F.records(codes))
    assert np.array_equal(ws.cpu().numpy().astype(int) - 127, es.T)


@pytest.mark.parametrize("b,out", [(3, "f32"), (3, "bf16"), (100, "f32"), (700, "bf16"), (700, "fast")])
def test_products_of_large_weights(S, b, out):  # noqa: F811
    """Weights up to 1.75 x 2^127, activations that bring the results back into range."""
    n, m = 200, 300
    rng = np.random.default_rng(2)
    w = np.clip(large(rng, n, m, "f32"), -1.75 * 2.0 ** 127, 1.75 * 2.0 ** 127)
    x = R.bf16(rng.standard_normal((b, m)) * 2.0 ** -40)
    lay = S.DeviceLayerFp8(torch.from_numpy(w).float().cuda(), transposed=True)
    xq, wq = F.quantize(x, 1), F.quantize(w, 128)
    v, dv = R.product_values(xq[2], wq[2], m)
    if out == "fast":
        dv = dv + F.aligned(xq, wq)
    got = S.svdq_fp8_linear(dev_bf16(x), lay, out_dtype=torch.float32 if out == "f32" else torch.bfloat16, fast_sums=out == "fast")
    close(got, *R.epilogue(v, dv, out="f32" if out == "f32" else "bf16"))
