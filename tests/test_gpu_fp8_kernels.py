"""Each kernel of the 8-bit floating-point products, by name: the tests say which one
a shape takes (the library's own plan) and fail where the plan has moved away."""
import numpy as np
import pytest

from tests import epi_ref as R
from tests import fp8_ref as F
from tests.fp8_kernel import kernel
from tests.test_gpu_fp8 import ACTS, Layer, S, close, dev_bf16, i32, ragged, rows_like  # noqa: F401 (S: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

MODES = ("bf16", "f32", "fast")


def dtype_of(mode):
    return torch.float32 if mode == "f32" else torch.bfloat16


def rounding(mode):
    return "f32" if mode == "f32" else "bf16"


# ---------------------------------------------------------------------------
# grouped by expert
# ---------------------------------------------------------------------------

# experts, rows, m, n, rows behind the last expert's, and the kernel of each mode
GROUPED = [
    (2, 2000, 129, 1000, 0, ("tiles", "tiles", "tiles")),
    (3, 2000, 129, 1000, 9, ("tiles", "tiles", "tiles")),
    (65, 2000, 129, 1000, 0, ("tiles", "tiles", "tiles")),
    (16, 5000, 300, 520, 130, ("tiles", "tiles", "tiles")),
    (8, 3001, 1152, 520, 1, ("tiles", "tiles", "tiles")),
    (4, 5000, 129, 520, 3, ("tiles", "tiles", "big 1")),
    (2, 2300, 260, 300, 5, ("rows 4", "rows 4", "big 1")),
    (6, 180, 300, 70, 2, ("rows 2", "rows 2", "rows 2")),
]


@pytest.mark.parametrize("E,b,m,n,pad,which", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(S, E, b, m, n, pad, which, gather):  # noqa: F811
    rng = np.random.default_rng([E, b, m, n])
    X = Layer(S, m, n, E, bias=E % 2 == 0, seed=21)
    off = ragged(rng, E, b, pad)
    if E > 2:
        assert (np.diff(off) == 0).any()  # an expert without rows
    rows = 1234 if gather else b
    x = rows_like(rng, rows, m)
    src = rng.integers(0, rows, b) if gather else np.arange(b)
    if gather:
        src[[0, 5, 40, b - pad - 1]] = [-1, rows, 1 << 30, -(1 << 31)]  # rows that are not there
        src[200 if b > 300 else 50] = src[100 if b > 300 else 51]
    gone = np.where((src >= 0)[:, None] & (src < rows)[:, None], x[np.clip(src, 0, rows - 1)], 0)
    live = np.zeros(b, bool)
    live[off[0]: off[-1]] = True
    dead = torch.from_numpy(~live).cuda()
    act, begin = ACTS[1 + E % 4], (0 if E % 3 else n // 3)
    qx, asc = S.svdq_fp8_quantize_act(dev_bf16(x))
    index = i32(src) if gather else None
    # of an expert with many rows the reference takes some: its ends and others
    some = {}
    for e in range(E):
        r = np.arange(off[e], off[e + 1])
        some[e] = r if len(r) <= 80 else np.unique(np.concatenate([r[:20], r[-20:], rng.choice(r, 60)]))
    ref = {e: X.product(gone[r], e) for e, r in some.items() if len(r)}
    more = {e: F.aligned(F.quantize(gone[r], 1), (X.codes[e], X.es[e], X.val[e])) for e, r in some.items() if len(r)}
    for mode, name in zip(MODES, which):
        assert kernel(b, n, m, E, mode) == name, mode
        y0 = torch.full((b, n + 5), 99.0, dtype=dtype_of(mode)).cuda()
        got = S.svdq_fp8_grouped_linear(dev_bf16(x), i32(off), X.layer, index, act=act, act_begin=begin, y=y0[:, 3: 3 + n],
                                        fast_sums=mode == "fast")
        for e, (v, dv) in ref.items():
            y, bound = R.epilogue(v, dv + more[e] if mode == "fast" else dv, act, begin, out=rounding(mode))
            close(got[torch.from_numpy(some[e]).cuda()], y, bound, (mode, e))
        assert (got[dead] == 99).all() and (y0[:, :3] == 99).all() and (y0[:, 3 + n:] == 99).all()
        assert not (got[~dead] == 99).all(1).any()
        y2 = torch.full((b, n), 99.0, dtype=dtype_of(mode)).cuda()
        S.svdq_fp8_grouped_gemm(qx, asc, i32(off), X.layer, index, act=act, act_begin=begin, y=y2, fast_sums=mode == "fast")
        assert torch.equal(y2, got)


@pytest.mark.parametrize("E,b,m,n,which", [(4, 2000, 129, 1000, ("tiles", "tiles", "tiles")), (4, 5000, 129, 520, ("tiles", "tiles", "big 1"))])
def test_offsets_of_any_content(S, E, b, m, n, which):  # noqa: F811
    """Offsets that are negative, too large or decreasing lead nowhere out of the rows."""
    X = Layer(S, m, n, E, seed=22)
    x = dev_bf16(rows_like(np.random.default_rng(b), b, m))
    for mode, name in zip(MODES, which):
        assert kernel(b, n, m, E, mode) == name, mode
        guard = torch.full((b + 40, n), 3.0, dtype=dtype_of(mode)).cuda()
        for off in ([0, -5, b + 7, 2, b], [b, b, b, b, b], [1 << 30, 0, -(1 << 30), b, 1 << 30], [-9, -8, -7, -6, -5], [b + 1, 0, 3, 1, 5]):
            guard.fill_(3.0)
            S.svdq_fp8_grouped_linear(x, i32(off), X.layer, y=guard[20: 20 + b], fast_sums=mode == "fast")
            assert (guard[:20] == 3).all() and (guard[20 + b:] == 3).all(), (mode, off)
        # sorted but not from 0: the rows before the first expert's and behind the last one's are left as they were
        guard.fill_(3.0)
        S.svdq_fp8_grouped_linear(x, i32([2, 300, 300, 301, b - 1]), X.layer, y=guard[20: 20 + b], fast_sums=mode == "fast")
        assert (guard[20:22] == 3).all() and (guard[19 + b:] == 3).all()
        assert not (guard[22: 19 + b] == 3).all(1).any()


def test_grouped_nonfinite_rows_and_experts_stay_their_own(S):  # noqa: F811
    E, b, m, n = 3, 2000, 129, 1000
    X = Layer(S, m, n, E, bias=False, seed=23)
    rng = np.random.default_rng(0)
    off = np.array([0, 700, 1450, b])
    x = dev_bf16(rows_like(rng, b, m))
    for mode in MODES:
        assert kernel(b, n, m, E, mode) == "tiles"
        want = S.svdq_fp8_grouped_linear(x, i32(off), X.layer, out_dtype=dtype_of(mode), fast_sums=mode == "fast")
        x2 = x.clone()
        x2[699, 128], x2[700, 0] = float("inf"), float("nan")
        qw, ws = X.layer.qw.clone(), X.layer.wscale.clone()
        qw[2, 1, 256:384] = 0x7F  # a block of NaN: columns 256 .. 383 of the last expert
        lay = S.GroupedDeviceLayerFp8.from_tensors(E, m, n, qw, ws)
        got = S.svdq_fp8_grouped_linear(x2, i32(off), lay, out_dtype=dtype_of(mode), fast_sums=mode == "fast")
        bad = torch.zeros(b, n, dtype=torch.bool).cuda()
        bad[699:701] = True
        bad[1450:, 256:384] = True
        assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad]), mode


# ---------------------------------------------------------------------------
# one layer: few rows of wide and deep ones, and the forms that the others' shapes leave out
# ---------------------------------------------------------------------------

DENSE = [
    (1, 4096, 14336, ("rows 1", "rows 1", "rows 1")),
    (1, 16384, 7168, ("rows 1", "rows 1", "rows 1")),
    (16, 8192, 8192, ("rows 1", "rows 1", "rows 1")),
    (17, 640, 33024, ("small", "small", "small")),
    (33, 640, 65536, ("small", "small", "tiles")),
    (40, 4608, 4608, ("rows 4", "rows 4", "pieces")),
    (64, 4608, 12288, ("pieces", "pieces", "small")),
    (64, 8192, 33024, ("pieces", "pieces", "pieces")),
    (300, 4608, 700, ("rows 4", "rows 4", "pieces")),
    (129, 640, 33024, ("tiles", "tiles", "big 1")),
    (1100, 1152, 4608, ("small", "small", "small")),
    (2048, 1152, 4608, ("tiles", "tiles", "big 1")),
]


@pytest.mark.parametrize("b,m,n,which", DENSE)
def test_dense(S, b, m, n, which):  # noqa: F811
    """Codes made on the device; the reference takes some rows and columns."""
    gen = torch.Generator(device="cuda").manual_seed(b + m + n)
    G = -(-m // 128)
    qw = torch.randint(0, 0x7F, (G, n, 128), dtype=torch.uint8, device="cuda", generator=gen)
    qw |= torch.randint(0, 2, qw.shape, dtype=torch.uint8, device="cuda", generator=gen) << 7
    if m % 128:
        qw[-1, :, m % 128:] = 0
    ws = torch.randint(110, 121, (G, -(-n // 128)), dtype=torch.uint8, device="cuda", generator=gen)
    bias = torch.randn(n, device="cuda", generator=gen).bfloat16()
    lay = S.DeviceLayerFp8.from_tensors(m, n, qw, ws, bias)
    rng = np.random.default_rng(b)
    x = rows_like(rng, b, m)
    rows = np.unique(np.concatenate([[0, b - 1], rng.integers(0, b, 40)]))
    cols = np.unique(np.concatenate([[0, 1, 127, n - 1, n - 65], rng.integers(0, n, 60)]))
    w = F.VALUES[qw[:, cols].cpu().numpy()]  # [G][cols][128]
    es = ws.cpu().numpy().astype(int)[:, cols // 128] - 127  # [G][cols]
    val = (w * 2.0 ** es.astype(float)[..., None]).transpose(1, 0, 2).reshape(len(cols), -1)[:, :m]
    xq = F.quantize(x[rows], 1)
    v, dv = R.product_values(xq[2], val, m, bias=bias.float().cpu().numpy().astype(np.float64)[cols])
    gate = torch.randn(1, n, device="cuda", generator=gen).bfloat16()
    for mode, name in zip(MODES, which):
        assert kernel(b, n, m, 0, mode) == name, mode
        wide = torch.randn(b, n + 7, device="cuda", generator=gen).to(dtype_of(mode))
        res = wide[rows][:, cols + 3].float().cpu().numpy().astype(np.float64)
        ends = wide[:, :3].clone(), wide[:, 3 + n:].clone()
        more = F.aligned(xq, (None, es.T, val), w_by=1) if mode == "fast" else 0
        y, bound = R.epilogue(v, dv + more, "silu", 0, gate=gate.float().cpu().numpy().astype(np.float64)[:, cols], gate_rows=b,
                              residual=res, out=rounding(mode))
        own = wide[:, 3: 3 + n]
        S.svdq_fp8_linear(dev_bf16(x), lay, act="silu", gate=gate, residual=own, y=own, fast_sums=mode == "fast")
        close(own[rows][:, cols], y, bound, mode)
        assert torch.equal(wide[:, :3], ends[0]) and torch.equal(wide[:, 3 + n:], ends[1])


@pytest.mark.parametrize("b,m,n,mode,name", [(700, 4608, 384, "bf16", "pieces"), (700, 4608, 384, "f32", "pieces"),
                                             (300, 4608, 700, "fast", "pieces"), (2100, 1024, 4100, "fast", "big 1"),
                                             (2048, 1152, 4608, "bf16", "tiles")])
def test_graphs_on_two_streams(S, b, m, n, mode, name):  # noqa: F811
    """Two captured calls, each with a workspace of its own, replayed together on new inputs between eager calls."""
    assert kernel(b, n, m, 0, mode) == name
    fast = mode == "fast"
    w = (torch.randn(n, m, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) / m ** 0.5).bfloat16()
    lay = S.DeviceLayerFp8(w, transposed=True)
    xs = [dev_bf16(rows_like(np.random.default_rng([b, i]), b, m)) for i in range(6)]
    eager = lambda x: S.svdq_fp8_linear(x, lay, act="silu", out_dtype=dtype_of(mode), fast_sums=fast)
    want = [eager(x) for x in xs]
    torch.cuda.synchronize()
    calls = []
    for _ in range(2):
        x = xs[0].clone()
        y = torch.empty(b, n, dtype=dtype_of(mode)).cuda()
        ws = torch.empty(S.svdq_fp8_linear_workspace_size(b, m, n), dtype=torch.uint8).cuda()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.svdq_fp8_linear(x, lay, act="silu", y=y, workspace=ws, fast_sums=fast)
        calls.append((x, y, g, torch.cuda.Stream()))
    for i in range(0, 6, 2):
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
        assert torch.equal(eager(xs[i]), want[i])
