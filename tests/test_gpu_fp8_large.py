"""Codes and weights of more than 4 GB in every kernel of the 8-bit floating-point
products: channel blocks, experts and their weights behind 32-bit offsets."""
import numpy as np
import pytest

from tests import epi_ref as R
from tests import fp8_ref as F
from tests.fp8_kernel import kernel
from tests.test_gpu_fp8 import S, close, dev_bf16, rows_like  # noqa: F401 (S: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

M, N = 16384, 270000  # 4.4 GB of codes


@pytest.fixture(scope="module")
def codes():
    gen = torch.Generator(device="cuda").manual_seed(4)
    qw = torch.randint(0, 0x7F, (M // 128 * N * 128,), dtype=torch.uint8, device="cuda", generator=gen)
    ws = torch.randint(118, 121, (280000,), dtype=torch.uint8, device="cuda", generator=gen)
    yield qw, ws
    del qw, ws
    torch.cuda.empty_cache()


def values(qw, ws, cols):
    """[cols][m] of qw [G][n][128], ws [G][ceil(n / 128)]."""
    w = F.VALUES[qw[:, cols].cpu().numpy()]
    w *= 2.0 ** (ws[:, [c // 128 for c in cols]].cpu().numpy().astype(float) - 127)[..., None]
    return w.transpose(1, 0, 2).reshape(len(cols), -1)


def dtype_of(mode):
    return torch.float32 if mode == "f32" else torch.bfloat16


@pytest.mark.parametrize("b,mode,name", [(2, "bf16", "rows 1"), (2, "f32", "rows 1"), (40, "bf16", "small"), (100, "f32", "tiles"),
                                         (100, "bf16", "tiles"), (100, "fast", "tiles"), (140, "fast", "big 1")])
def test_channel_blocks(S, codes, b, mode, name):  # noqa: F811
    got = kernel(b, N, M, 0, mode)
    print(f"fp8 weights of 4.4 GB, {b} rows, {mode}: {got}", flush=True)
    assert got.split()[0] == name.split()[0]
    qw, ws = codes[0].view(M // 128, N, 128), codes[1][: M // 128 * -(-N // 128)].view(M // 128, -(-N // 128))
    lay = S.DeviceLayerFp8.from_tensors(M, N, qw, ws)
    x = rows_like(np.random.default_rng(13), b, M)
    y = S.svdq_fp8_linear(dev_bf16(x), lay, out_dtype=dtype_of(mode), fast_sums=mode == "fast")
    cols = [0, 1, 127, 128, 131072, 262143, 262144, N - 129, N - 1]
    rows = [0, b // 2, b - 1]
    w = values(qw, ws, cols)
    xq = F.quantize(x[rows], 1)
    v, dv = R.product_values(xq[2], w, M)
    if mode == "fast":
        es = ws.cpu().numpy().astype(int)[:, [c // 128 for c in cols]].T - 127
        dv = dv + F.aligned(xq, (None, es, w), w_by=1)
    close(y[rows][:, cols], *R.epilogue(v, dv, out="f32" if mode == "f32" else "bf16"))


@pytest.mark.parametrize("b,mode,name", [(60, "bf16", "rows 1"), (60, "f32", "rows 1"), (4000, "bf16", "tiles"), (4000, "f32", "tiles"),
                                         (4000, "fast", "tiles"), (70000, "fast", "big 1")])
def test_experts(S, codes, b, mode, name):  # noqa: F811
    """The last experts' weights, scales and biases lie 4 GB behind the first one's."""
    E, m, n = 60, 8192, 9000
    assert E * m * n > 1 << 32 and kernel(b, n, m, E, mode) == name
    qw, ws = codes[0][: E * m * n].view(E, m // 128, n, 128), codes[1][: E * (m // 128) * 71].view(E, m // 128, 71)
    bias = torch.randn(E, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    lay = S.GroupedDeviceLayerFp8.from_tensors(E, m, n, qw, ws, bias)
    rng = np.random.default_rng(6)
    tokens = min(b, 300)
    x = rows_like(rng, tokens, m)
    src = rng.integers(0, tokens, b)
    off = np.round(np.linspace(0, b, E + 1)).astype(int)
    y = S.svdq_fp8_grouped_linear(dev_bf16(x), torch.from_numpy(off.astype(np.int32)).cuda(), lay,
                                  torch.from_numpy(src.astype(np.int32)).cuda(), out_dtype=dtype_of(mode), fast_sums=mode == "fast")
    cols = [0, 1, 127, 128, 4500, n - 129, n - 1]
    for e in (0, 1, E // 2, E - 2, E - 1):
        rows = np.unique([off[e], (off[e] + off[e + 1]) // 2, off[e + 1] - 1])
        w = values(qw[e], ws[e], cols)
        xq = F.quantize(x[src[rows]], 1)
        v, dv = R.product_values(xq[2], w, m, bias=bias[e, cols].float().cpu().numpy().astype(np.float64))
        if mode == "fast":
            es = ws[e].cpu().numpy().astype(int)[:, [c // 128 for c in cols]].T - 127
            dv = dv + F.aligned(xq, (None, es, w), w_by=1)
        close(y[rows][:, cols], *R.epilogue(v, dv, out="f32" if mode == "f32" else "bf16"), e)


@pytest.mark.parametrize("transposed", [False, True])
def test_quantizing_many_weights(S, transposed):  # noqa: F811
    """W, its codes and its scales of experts past 4 GB (of W: 8.9 GB in bf16)."""
    E, m, n = 60, 8192, 9000
    shape = (E, n, m) if transposed else (E, m, n)
    w = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    for e in range(E):
        w[e] = torch.randn(shape[1:], device="cuda", generator=gen).bfloat16()
    qw, ws = S.svdq_fp8_quantize_weights(w, transposed=transposed)
    for e in (0, E // 2, E - 1):
        one = S.svdq_fp8_quantize_weights(w[e].contiguous(), transposed=transposed)
        assert torch.equal(qw[e], one[0]) and torch.equal(ws[e], one[1]), e
    part = w[E - 1][-384:].float().cpu().numpy().astype(np.float64)  # W^T: the last columns; W: the last channels
    if transposed:  # 9000 = 70 x 128 + 40: columns 8960 .. 8999 are the last block
        c, es, _ = F.quantize(part[-40:, :256], 128)
        assert np.array_equal(qw[E - 1, :2, -40:].cpu().numpy(), F.records(c))
        assert np.array_equal(ws[E - 1, :2, -1].cpu().numpy().astype(int) - 127, es[0])
    else:
        c, es, _ = F.quantize(part[-128:, :256].T, 128)
        assert np.array_equal(qw[E - 1, -1, :256].cpu().numpy(), F.records(c)[0])
        assert np.array_equal(ws[E - 1, -1, :2].cpu().numpy().astype(int) - 127, es[:, 0])
