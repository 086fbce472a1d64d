"""The gradient of an 8-bit floating-point layer's input (the layer of the transposed
weight) against differences of the layer, exactly."""
import numpy as np
import pytest

from tests import fp8_ref as F
from tests.fp8_kernel import kernel
from tests.test_gpu_fp8 import S, dev_bf16, to_np  # noqa: F401 (S: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def grid(rng, shape):
    """Multiples of 1 / 8 below 2 whose blocks' largest magnitude is 1.875: codes stand for them as they are."""
    v = rng.integers(-15, 16, shape) / 8.0
    v[..., ::128] = 1.875
    return v


@pytest.mark.parametrize("b,m,n", [(1, 300, 200), (5, 1000, 130), (70, 640, 300), (700, 384, 1500)])
def test_input_gradient_is_the_difference(S, b, m, n):  # noqa: F811
    """X, W and dY on a grid that their codes hold: every product is a multiple of 1 / 64 and every sum below
    1500 x 1.875^2 < 2^13, so 32 bits hold all of them whatever their order, and the change of <dY, Y> along one entry of
    X is the gradient's entry, not only nearly."""
    print(f"fp8 gradient b={b} m={m} n={n}: {kernel(b, n, m, 0, 'f32')}, {kernel(b, m, n, 0, 'f32')}", flush=True)
    rng = np.random.default_rng([b, m, n])
    w, x, dy = grid(rng, (m, n)), grid(rng, (b, m)), grid(rng, (b, n))
    assert (F.quantize(w.T, 128)[2] == w.T).all() and (F.quantize(x[:1], 1)[2] == x[:1]).all()
    wd = torch.from_numpy(w).float().cuda()
    fwd, bwd = S.DeviceLayerFp8(wd), S.DeviceLayerFp8(wd, transposed=True)
    g = to_np(S.svdq_fp8_linear(dev_bf16(dy), bwd, out_dtype=torch.float32))
    assert np.array_equal(g, dy @ w.T)  # the formula
    run = lambda v: to_np(S.svdq_fp8_linear(dev_bf16(v), fwd, out_dtype=torch.float32))
    for i, j in [(0, 1), (b // 2, 77), (b - 1, 129), (b - 1, m - 1), (b // 3, 260)]:
        lo, hi = x.copy(), x.copy()
        lo[i, j], hi[i, j] = -1.0, 1.0
        assert float(((run(hi) - run(lo)) * dy).sum()) / 2 == g[i, j], (i, j)
