"""The 8-bit floating-point setting on the GPU against 64-bit references: codes
and scales bit for bit, products within the derived bounds of tests/fp8_ref.py."""
import sys

import numpy as np
import pytest

from tests import epi_ref as R
from tests import fp8_ref as F

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ACTS = ("none", "gelu_tanh", "gelu_erf", "silu", "relu")


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a4_rank_corrected_amd as S
    S.lib()
    return S


def dev_bf16(v):
    return torch.from_numpy(R.bf16_bits(v).view(np.int16)).cuda().view(torch.bfloat16)


def to_np(y):
    return y.float().cpu().numpy().astype(np.float64)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32).cuda()


def dtype_of(out):
    return torch.float32 if out == "f32" else torch.bfloat16


def close(y, ref, bound, what=""):
    y = to_np(y)
    bad = ~(np.abs(y - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3], y[bad][:3], ref[bad][:3], bound[bad][:3])


def rows_like(rng, b, m):
    x = rng.standard_normal((b, m)) * np.exp(0.7 * rng.standard_normal((b, 1)))
    x[:, rng.choice(m, max(1, m // 60), replace=False)] *= 30
    return R.bf16(x)


class Layer:
    """A random layer (or one per expert): 64-bit values of its codes, and the library's."""

    def __init__(self, S, m, n, E=0, bias=True, seed=0, transposed=True, dtype=torch.bfloat16):
        rng = np.random.default_rng([seed, m, n, E])
        w = rng.standard_normal((max(E, 1), n, m)) / np.sqrt(m) * np.exp(0.4 * rng.standard_normal((max(E, 1), n, 1)))
        w = R.bf16(w) if dtype == torch.bfloat16 else w.astype(np.float32).astype(np.float64)
        q = [F.quantize(v, 128) for v in w]
        self.m, self.n, self.E, self.w = m, n, E, w
        self.codes, self.es, self.val = ([v[i] for v in q] for i in range(3))
        self.bias = R.bf16(0.5 * rng.standard_normal((max(E, 1), n))) if bias else None
        wd = torch.from_numpy(w if transposed else np.ascontiguousarray(w.transpose(0, 2, 1))).to(dtype).cuda()
        bd = dev_bf16(self.bias) if bias else None
        if E:
            self.layer = S.GroupedDeviceLayerFp8(wd, bd, transposed=transposed)
        else:
            self.layer = S.DeviceLayerFp8(wd[0], None if bd is None else bd[0], transposed=transposed)

    def product(self, x, e=0, tiles=False):
        """(v, bound) of rows x (bf16 values); tiles: by the 8-bit matrix instruction."""
        xq = F.quantize(x, 1)
        v, dv = R.product_values(xq[2], self.val[e], self.m, bias=None if self.bias is None else self.bias[e])
        if tiles:
            dv = dv + F.aligned(xq, (self.codes[e], self.es[e], self.val[e]))
        return v, dv


# ---------------------------------------------------------------------------
# quantization
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("b,m", [(1, 1), (1, 128), (3, 127), (16, 129), (17, 1000), (5, 513), (40, 1152), (2, 4103)])
def test_act_codes(S, b, m):
    _say(f"fp8 act b={b} m={m}")
    rng = np.random.default_rng([b, m])
    x = rows_like(rng, b, m)
    x[b // 2] = 0
    if m > 128:
        x[0, 3] = R.bf16(448 * 2.0 ** -5)  # borders of a block's scale
        x[b - 1, :128] = R.bf16(np.array(2.0 ** -133))
    qx, asc = S.svdq_fp8_quantize_act(dev_bf16(x))
    codes, es, _ = F.quantize(x, 1)
    assert np.array_equal(qx.cpu().numpy(), F.records(codes))
    assert np.array_equal(asc.cpu().numpy().astype(int) - 127, es.T)


def test_every_bf16_value(S):
    """Every finite bf16 magnitude, both signs, as a block's maximum and below a larger one."""
    bits = np.arange(0x7F80, dtype=np.uint16)
    v = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    x = np.zeros((len(v), 128))
    x[:, 0] = v
    x[:, 1] = -v
    for c, f in enumerate((0.5, 0.3, 0.071, 0.0021, 0.00037, 1.0 / 448), start=2):
        x[:, c] = R.bf16(v * f)
    x[:, 9] = -0.0
    qx, asc = S.svdq_fp8_quantize_act(dev_bf16(x))
    f, k = np.frexp(v)
    es = np.where(v > 0, np.maximum(k - np.where(f <= 0.875, 9, 8), -126), -126)
    assert np.array_equal(asc.cpu().numpy()[0].astype(int) - 127, es)
    codes = F.encode(x * 2.0 ** -es.astype(np.float64)[:, None])
    got = qx.cpu().numpy()[0]
    bad = np.argwhere(got != codes)
    assert not len(bad), (len(bad), [(hex(bits[i]), int(c), hex(got[i, c]), hex(codes[i, c])) for i, c in bad[:6]])


def test_act_nonfinite_blocks(S):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((20, 300)).astype(np.float64)
    x = R.bf16(x)
    x[3, 7], x[4, 140], x[5, 299], x[6, 0] = np.inf, np.nan, -np.inf, -np.nan
    xd = dev_bf16(np.nan_to_num(x, nan=0, posinf=0, neginf=0))
    for i, j in ((3, 7), (4, 140), (5, 299), (6, 0)):
        xd[i, j] = float(x[i, j])
    qx, asc = S.svdq_fp8_quantize_act(xd)
    codes, es, _ = F.quantize(x, 1)
    want = F.records(codes)
    got = qx.cpu().numpy().copy()
    got[2, 5, 300 - 256:] = 0  # codes behind the last channel of a block of NaN: any
    want[2, 5, 300 - 256:] = 0
    assert np.array_equal(got, want)
    assert np.array_equal(asc.cpu().numpy().astype(int) - 127, es.T)


@pytest.mark.parametrize("E,m,n", [(0, 1, 1), (0, 128, 128), (0, 130, 257), (0, 300, 77), (3, 129, 200), (2, 1000, 130)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transposed", [False, True])
def test_weight_codes(S, E, m, n, dtype, transposed):
    _say(f"fp8 weights E={E} m={m} n={n} {dtype} transposed={transposed}")
    X = Layer(S, m, n, E, seed=1, transposed=transposed, dtype=dtype)
    qw, ws = X.layer.qw.cpu().numpy(), X.layer.wscale.cpu().numpy().astype(int) - 127
    for e in range(max(E, 1)):
        q, s = (qw[e], ws[e]) if E else (qw, ws)
        assert np.array_equal(q, F.records(X.codes[e])), e
        assert np.array_equal(s, X.es[e].T), e


def test_weight_extremes(S):
    """Blocks of zeros, of fp32 subnormals, of the largest values, of infinities; unaligned W."""
    w = np.zeros((400, 290), np.float32)
    rng = np.random.default_rng(3)
    w[:128, 128:256] = rng.standard_normal((128, 128)) * 1e-41
    w[128:256, :128] = rng.standard_normal((128, 128)) * 1e38
    w[256:384, 128:256] = rng.standard_normal((128, 128)) * 2.0 ** -20
    w[390, 5] = np.inf
    w[395, 200] = np.nan
    flat = torch.zeros(w.size + 1).cuda()
    flat[1:] = torch.from_numpy(w.reshape(-1)).cuda()
    qw, ws = S.svdq_fp8_quantize_weights(flat[1:].view(400, 290), transposed=True)
    codes, es, _ = F.quantize(w, 128)
    got, want = qw.cpu().numpy(), F.records(codes)
    assert np.array_equal(got, want), np.argwhere(got != want)[:4]
    assert np.array_equal(ws.cpu().numpy().astype(int) - 127, es.T)


def test_transposed_layer_has_the_same_values(S):
    """The codes of W and of its transpose stand for one matrix: the gradient of a layer's input is the layer of W^T."""
    rng = np.random.default_rng(8)
    m, n, b = 300, 200, 70
    w = torch.from_numpy(rng.standard_normal((m, n)) / 10).float().cuda()
    fwd, bwd = S.DeviceLayerFp8(w), S.DeviceLayerFp8(w, transposed=True)  # m -> n, and n -> m of W^T
    cf, cb = fwd.qw.cpu().numpy(), bwd.qw.cpu().numpy()
    assert np.array_equal(cf.transpose(1, 0, 2).reshape(n, -1)[:, :m], cb.transpose(1, 0, 2).reshape(m, -1)[:, :n].T)
    assert np.array_equal(fwd.wscale.cpu().numpy(), bwd.wscale.cpu().numpy().T)
    # dX = dY W^T: against the formula, and y's change along a direction (bilinear in x: a difference is exact but
    # for the quantization of the two rows, so equal rows of codes are taken)
    val = F.quantize(w.cpu().numpy().T.astype(np.float64), 128)[2]  # [n][m]
    dy = rows_like(rng, b, n)
    v, dv = R.product_values(F.quantize(dy, 1)[2], val.T, n)
    y, bound = R.epilogue(v, dv)
    dx = S.svdq_fp8_linear(dev_bf16(dy), bwd, out_dtype=torch.float32)
    close(dx, y, bound, "dx")
    # against differences: x on a grid that quantization keeps (steps of 1 / 8 below 2), one channel moved
    x = rng.integers(-15, 16, (1, m)) / 8.0
    x[0, ::128] = 1.875  # the blocks' maxima stay
    d = F.quantize(R.bf16(rng.standard_normal((1, n))), 1)[2]
    g = to_np(S.svdq_fp8_linear(dev_bf16(d), bwd, out_dtype=torch.float32))[0]
    for j in (1, 77, 129, m - 1):
        lo, hi = x.copy(), x.copy()
        lo[0, j], hi[0, j] = -1.0, 1.0
        yl, yh = (to_np(S.svdq_fp8_linear(dev_bf16(t), fwd, out_dtype=torch.float32))[0] for t in (lo, hi))
        diff = float(((yh - yl) * d[0]).sum() / 2)
        scale = float(np.abs(x).sum() * np.abs(val).max() * np.abs(d).sum())
        assert abs(diff - g[j]) <= (m + n + 48) * 4 * R.U * scale, (j, diff, g[j])


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

# one row and a few (quantized in the product's kernel or before it), the row kernel, tiles of 64 x 128, whole and split
# ones of 128 x 128, tiles of 256 x 256 with a last round whole, in halves and in quarters
SHAPES = [(1, 1, 1), (1, 8192, 40), (1, 8193, 40), (4, 2048, 33), (9, 900, 20), (16, 512, 70), (17, 128, 50), (40, 100, 90), (1, 128, 16), (1, 1152, 700), (2, 130, 33), (7, 1000, 513), (16, 256, 128), (17, 384, 130), (33, 700, 64),
          (64, 2048, 96), (65, 129, 257), (130, 640, 300), (257, 1152, 200), (300, 4200, 72), (512, 300, 520),
          (333, 1000, 1500), (450, 1900, 900), (2100, 640, 900), (2048, 130, 257), (2300, 400, 513), (2500, 1100, 300),
          (300, 4608, 700), (400, 4700, 1100), (129, 8192, 1000), (4100, 140, 2300), (4608, 130, 4800), (4350, 260, 4150), (4096, 128, 4096)]


@pytest.mark.parametrize("b,m,n", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear(S, b, m, n, out):
    _say(f"fp8 linear b={b} m={m} n={n} {out}")
    rng = np.random.default_rng([b, m, n])
    X = Layer(S, m, n, bias=b % 2 == 1, seed=2)
    x = rows_like(rng, b, m)
    x[b // 2] = 0
    v, dv = X.product(x, tiles=out == "bf16" and b > 64)
    act, begin = ACTS[(b + n) % 5], (n // 3 if n % 2 else 0)
    y, bound = R.epilogue(v, dv, act, begin, out=out)
    xd = dev_bf16(x)
    got = S.svdq_fp8_linear(xd, X.layer, act=act, act_begin=begin, out_dtype=dtype_of(out))
    close(got, y, bound)
    qx, asc = S.svdq_fp8_quantize_act(xd)
    two = S.svdq_fp8_gemm(qx, asc, X.layer, act=act, act_begin=begin, out_dtype=dtype_of(out))
    assert torch.equal(got, two)


@pytest.mark.parametrize("b", [1, 40, 200, 2049])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,begin", [(150, 31), (256, 128), (512, 0), (256, 200)])
def test_epilogue(S, b, act, n, begin):
    """Gate, residual and strides, each with an activation; nothing is written between the rows."""
    m = 384
    rng = np.random.default_rng([b, 7])
    X = Layer(S, m, n, seed=3)
    x = rows_like(rng, b, m)
    rows = max(1, b // 3)
    gate = R.bf16(rng.standard_normal((-(-b // rows), n)))
    for out in ("f32", "bf16"):
        res = rng.standard_normal((b, n))
        res = R.bf16(res) if out == "bf16" else res.astype(np.float32).astype(np.float64)
        v, dv = X.product(x, tiles=out == "bf16" and b > 64)
        y, bound = R.epilogue(v, dv, act, begin, gate=gate, gate_rows=rows, residual=res, out=out)
        wide = torch.full((b, n + 9), 5.0, dtype=dtype_of(out)).cuda()
        wres = torch.full((b, n + 3), 7.0, dtype=dtype_of(out)).cuda()
        wres[:, 2: 2 + n] = torch.from_numpy(res).to(dtype_of(out)).cuda()
        got = S.svdq_fp8_linear(dev_bf16(x), X.layer, act=act, act_begin=begin, gate=dev_bf16(gate), gate_rows=rows,
                                residual=wres[:, 2: 2 + n], y=wide[:, 5: 5 + n])
        close(got, y, bound, out)
        assert (wide[:, :5] == 5).all() and (wide[:, 5 + n:] == 5).all()
        # in place on the residual
        own = wres[:, 2: 2 + n]
        S.svdq_fp8_linear(dev_bf16(x), X.layer, act=act, act_begin=begin, gate=dev_bf16(gate), gate_rows=rows, residual=own, y=own)
        assert torch.equal(own, got)
        assert (wres[:, :2] == 7).all() and (wres[:, 2 + n:] == 7).all()


@pytest.mark.parametrize("act,n,begin", [("gelu_tanh", 512, 0), ("silu", 450, 200), ("relu", 512, 128)])
def test_epilogue_of_larger_tiles(S, act, n, begin):
    test_epilogue(S, 4200, act, n, begin)


@pytest.mark.parametrize("b", [1, 5, 64, 300])
def test_in_place_on_its_input(S, b):
    m = n = 256
    X = Layer(S, m, n, seed=4)
    x = dev_bf16(rows_like(np.random.default_rng(b), b, m))
    want = S.svdq_fp8_linear(x, X.layer, act="silu", residual=x)
    got = S.svdq_fp8_linear(x, X.layer, act="silu", residual=x, y=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("b", [1, 20, 200])
def test_unaligned_operands(S, b):
    """x, scales, bias and gate at any element's address, odd m and n."""
    m, n = 333, 77
    rng = np.random.default_rng(b)
    X = Layer(S, m, n, seed=5)
    x = rows_like(rng, b, m)
    flat = torch.zeros(b * m + 1, dtype=torch.bfloat16).cuda()
    flat[1:] = dev_bf16(x).reshape(-1)
    ws = torch.zeros(X.layer.wscale.numel() + 1, dtype=torch.uint8).cuda()
    ws[1:] = X.layer.wscale.reshape(-1)
    bias = torch.zeros(n + 1, dtype=torch.bfloat16).cuda()
    bias[1:] = X.layer.bias
    gate = torch.zeros(n + 1, dtype=torch.bfloat16).cuda()
    gate[1:] = 0.5
    lay = S.DeviceLayerFp8.from_tensors(m, n, X.layer.qw, ws[1:].view(X.layer.wscale.shape), bias[1:])
    v, dv = X.product(x)
    y, bound = R.epilogue(v, dv, "silu", gate=np.full((1, n), 0.5))
    got = S.svdq_fp8_linear(flat[1:].view(b, m), lay, act="silu", gate=gate[1:].view(1, n), out_dtype=torch.float32)
    close(got, y, bound)
    qx, asc = S.svdq_fp8_quantize_act(dev_bf16(x))
    off = torch.zeros(asc.numel() + 1, dtype=torch.uint8).cuda()
    off[1:] = asc.reshape(-1)
    got2 = S.svdq_fp8_gemm(qx, off[1:].view(asc.shape), lay, act="silu", gate=gate[1:].view(1, n), out_dtype=torch.float32)
    assert torch.equal(got, got2)


@pytest.mark.parametrize("b,out", [(3, "f32"), (70, "f32"), (300, "f32"), (70, "bf16"), (300, "bf16"), (2100, "bf16")])
def test_nonfinite_rows_and_columns_stay_their_own(S, b, out):
    m, n = 640, 300
    rng = np.random.default_rng(b)
    w = torch.from_numpy(rng.standard_normal((n, m)) / 25).bfloat16().cuda()
    x = dev_bf16(rows_like(rng, b, m))
    want = S.svdq_fp8_linear(x, S.DeviceLayerFp8(w, transposed=True), out_dtype=dtype_of(out))
    x2, w2 = x.clone(), w.clone()
    x2[b // 2, 600] = float("inf")
    w2[130, 5] = float("nan")  # columns 128 .. 255
    got = S.svdq_fp8_linear(x2, S.DeviceLayerFp8(w2, transposed=True), out_dtype=dtype_of(out))
    bad = torch.zeros(b, n, dtype=torch.bool).cuda()
    bad[b // 2] = True
    bad[:, 128:256] = True
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], want[~bad])


def test_b0(S):
    X = Layer(S, 200, 30, seed=6)
    x = torch.empty(0, 200, dtype=torch.bfloat16).cuda()
    assert S.svdq_fp8_linear(x, X.layer).shape == (0, 30)
    qx, asc = S.svdq_fp8_quantize_act(x)
    assert qx.shape == (2, 0, 128) and asc.shape == (2, 0)
    assert S.svdq_fp8_gemm(qx, asc, X.layer).shape == (0, 30)


@pytest.mark.parametrize("rows,out", [(6, "f32"), (100, "f32"), (100, "bf16"), (2100, "bf16")])
def test_extreme_scales(S, rows, out):
    """Scales far apart within a row and a product near the ends of fp32's range."""
    m, n = 512, 40
    rng = np.random.default_rng(11)
    w = rng.standard_normal((n, m)) / 20
    w[:, 128:256] *= 2.0 ** 40
    w[:, 256:384] *= 2.0 ** -60
    w = R.bf16(w)
    x = rng.standard_normal((6, m))
    x[:, 128:256] *= 2.0 ** -40
    x[1] *= 2.0 ** 60
    x[2] *= 2.0 ** -60
    x[3, :128] *= 2.0 ** 100
    x = R.bf16(x)
    lay = S.DeviceLayerFp8(dev_bf16(w), transposed=True)
    x = np.tile(x, (-(-rows // 6), 1))[:rows]
    xq, wq = F.quantize(x, 1), F.quantize(w, 128)
    v, dv = R.product_values(xq[2], wq[2], m)
    if out == "bf16":
        dv = dv + F.aligned(xq, wq)
    close(S.svdq_fp8_linear(dev_bf16(x), lay, out_dtype=dtype_of(out)), *R.epilogue(v, dv, out=out))


@pytest.mark.parametrize("rows,out", [(4, "f32"), (6, "bf16"), (100, "f32"), (2100, "bf16")])
def test_ends_of_the_range(S, rows, out):
    """The least scales of W (weights down to 2^-135) beside the largest of X.  As bf16 a weight is off by half a
    step of 2^-133 at most."""
    m, n = 384, 300
    rng = np.random.default_rng(17)
    w = rng.standard_normal((n, m)) * 2.0 ** -120 * np.exp2(-16.0 * rng.random((n, m)))
    w[:, :128] = rng.integers(-20, 20, (n, 128)) * 2.0 ** -135
    w = w.astype(np.float32).astype(np.float64)
    x = rng.standard_normal((6, m)) * 2.0 ** 124
    x[3] = rng.uniform(-1.9, 1.9, m) * 2.0 ** 127
    x = R.bf16(x)
    x = np.tile(x, (-(-rows // 6), 1))[:rows]
    lay = S.DeviceLayerFp8(torch.from_numpy(w).float().cuda(), transposed=True)
    xq, wq = F.quantize(x, 1), F.quantize(w, 128)
    assert wq[1].min() == -126 and xq[1].max() == 120
    v, dv = R.product_values(xq[2], wq[2], m)
    dv = dv + 2.0 ** -134 * np.abs(xq[2]).sum(1, keepdims=True)
    if out == "bf16":
        dv = dv + F.aligned(xq, wq)
    close(S.svdq_fp8_linear(dev_bf16(x), lay, out_dtype=dtype_of(out)), *R.epilogue(v, dv, out=out))


# ---------------------------------------------------------------------------
# grouped by expert
# ---------------------------------------------------------------------------

def ragged(rng, E, b, pad):
    c = np.diff(np.concatenate([[0], np.sort(rng.integers(0, b - pad + 1, E - 1)), [b - pad]]))
    if E > 2:
        c[0], c[E // 2] = c[0] + c[E // 2], 0  # an expert without rows
    return np.concatenate([[0], np.cumsum(c)])


GROUPED = [(1, 1, 64, 1, 0), (1, 30, 130, 70, 0), (3, 5, 200, 33, 0), (4, 70, 1024, 130, 9), (8, 300, 640, 200, 0),
           (64, 90, 128, 40, 5), (65, 300, 300, 24, 0), (5, 700, 256, 300, 3), (3, 900, 129, 150, 0), (2, 2300, 260, 300, 5), (1024, 700, 64, 8, 0)]


@pytest.mark.parametrize("E,b,m,n,pad", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped(S, E, b, m, n, pad, gather, out):
    _say(f"fp8 grouped E={E} b={b} m={m} n={n} pad={pad} gather={gather} {out}")
    rng = np.random.default_rng([E, b, m, n])
    X = Layer(S, m, n, E, bias=E % 2 == 1, seed=7)
    off = ragged(rng, E, b, pad)
    rows = 23 if gather else b
    x = rows_like(rng, rows, m)
    src = rng.integers(0, rows, b) if gather else np.arange(b)
    if gather and b > 4:
        src[:4] = [-1, rows, 1 << 30, src[4]]  # rows that are not there, and one row twice
    y0 = torch.full((b, n + 3), 99.0, dtype=dtype_of(out)).cuda()
    act, begin = ACTS[E % 5], n // 4
    got = S.svdq_fp8_grouped_linear(dev_bf16(x), i32(off), X.layer, i32(src) if gather else None, act=act, act_begin=begin,
                                    y=y0[:, 1: 1 + n])
    gone = np.where((src >= 0)[:, None] & (src < rows)[:, None], x[np.clip(src, 0, rows - 1)], 0)
    live = np.zeros(b, bool)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        live[s] = True
        v, dv = X.product(gone[s], e, tiles=out == "bf16" and b > 64 * E)
        y, bound = R.epilogue(v, dv, act, begin, out=out)
        close(got[s], y, bound, e)
    assert (got[torch.from_numpy(~live).cuda()] == 99).all()
    assert (y0[:, 0] == 99).all() and (y0[:, n + 1:] == 99).all()
    qx, asc = S.svdq_fp8_quantize_act(dev_bf16(x))
    y2 = torch.full((b, n), 99.0, dtype=dtype_of(out)).cuda()
    S.svdq_fp8_grouped_gemm(qx, asc, i32(off), X.layer, i32(src) if gather else None, act=act, act_begin=begin, y=y2)
    assert torch.equal(y2, got)


@pytest.mark.parametrize("b", [6, 150, 900])
def test_offsets_of_any_content(S, b):
    """Offsets that are negative, too large or decreasing lead nowhere out of the rows."""
    E, m, n = 4, 200, 40
    X = Layer(S, m, n, E, seed=9)
    x = dev_bf16(rows_like(np.random.default_rng(b), b, m))
    guard = torch.full((b + 40, n), 3.0).cuda()
    for off in ([0, -5, b + 7, 2, b], [b, b, b, b, b], [1 << 30, 0, -(1 << 30), b, 1 << 30], [-9, -8, -7, -6, -5],
                [b + 1, 0, 3, 1, 5]):
        guard.fill_(3.0)
        S.svdq_fp8_grouped_linear(x, i32(off), X.layer, y=guard[20: 20 + b])
        assert (guard[:20] == 3).all() and (guard[20 + b:] == 3).all(), off
    # sorted but not from 0: the rows before the first expert's are left as they were
    guard.fill_(3.0)
    S.svdq_fp8_grouped_linear(x, i32([2, 3, 3, 4, b - 1]), X.layer, y=guard[20: 20 + b])
    assert (guard[20:22] == 3).all() and (guard[19 + b:] == 3).all() and not (guard[22: 19 + b] == 3).any()


# ---------------------------------------------------------------------------
# streams, graphs, sizes
# ---------------------------------------------------------------------------

def test_same_inputs_same_bits_and_side_stream(S):
    X = Layer(S, 1152, 640, seed=10)
    side = torch.cuda.Stream()
    for b in (1, 48, 260, 2200):
        x = dev_bf16(rows_like(np.random.default_rng(b), b, 1152))
        want = S.svdq_fp8_linear(x, X.layer, act="gelu_tanh")
        torch.cuda.synchronize()
        for _ in range(3):
            assert torch.equal(S.svdq_fp8_linear(x, X.layer, act="gelu_tanh"), want)
        y = S.svdq_fp8_linear(x, X.layer, act="gelu_tanh", stream=side)
        side.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("b,m", [(1, 1024), (40, 1024), (300, 1024), (300, 4608), (2100, 1024)])
def test_graphs_on_two_streams(S, b, m):
    """Two captured calls, each with a workspace of its own, replayed together on new inputs."""
    n = 4100 if b > 2000 else (700 if m > 4000 else 200)
    X = Layer(S, m, n, seed=12)
    xs = [dev_bf16(rows_like(np.random.default_rng([b, i]), b, m)) for i in range(8)]
    want = [S.svdq_fp8_linear(x, X.layer, act="silu") for x in xs]
    torch.cuda.synchronize()
    calls = []
    for _ in range(2):
        x = xs[0].clone()
        y = torch.empty(b, n, dtype=torch.bfloat16).cuda()
        ws = torch.empty(S.svdq_fp8_linear_workspace_size(b, m, n), dtype=torch.uint8).cuda()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.svdq_fp8_linear(x, X.layer, act="silu", y=y, workspace=ws)
        calls.append((x, y, g, torch.cuda.Stream()))
    for i in range(0, 8, 2):
        for k, (x, y, g, st) in enumerate(calls):
            x.copy_(xs[i + k])
            y.zero_()
        torch.cuda.synchronize()
        for x, y, g, st in calls:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for k, (x, y, g, st) in enumerate(calls):
            assert torch.equal(y, want[i + k]), (i, k)


def test_codes_past_32_bit_offsets(S):
    """Weights of more than 4 GB: channel blocks and experts lie behind 32-bit offsets."""
    m, n, b = 16384, 270000, 2
    _say("fp8 weights of 4.4 GB")
    qw = torch.randint(0, 0x7F, (m // 128, n, 128), dtype=torch.uint8, device="cuda")
    ws = torch.randint(118, 121, (m // 128, -(-n // 128)), dtype=torch.uint8, device="cuda")
    lay = S.DeviceLayerFp8.from_tensors(m, n, qw, ws)
    x = rows_like(np.random.default_rng(13), b, m)
    got = S.svdq_fp8_linear(dev_bf16(x), lay, out_dtype=torch.float32)
    cols = [0, 1, 127, 128, 131072, 262143, 262144, n - 129, n - 1]
    w = F.VALUES[qw[:, cols].cpu().numpy()]  # [G][cols][128]
    w *= 2.0 ** (ws[:, [c // 128 for c in cols]].cpu().numpy().astype(float) - 127)[..., None]
    w = w.transpose(1, 0, 2).reshape(len(cols), m)
    close(got[:, cols], *R.epilogue(*R.product_values(F.quantize(x, 1)[2], w, m)))
