"""Products with an epilogue, the forms that differ between the settings and
between their kernels (row kernel, whole tiles, pieces of tiles and their
reduction): slices, unaligned operands, rows and columns that are not finite,
every block scale, and the 8-bit product on both sides of the choice between
small tiles and pieces."""
import numpy as np
import pytest

from tests import epi_ref as R
from tests import layout as LY
from tests.test_gpu_epilogue import ACTS, E2M1, Case, S, _say, dev, to_np  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# (setting, b, m): the row kernel's three block sizes, whole tiles, pieces
FORMS = [("int4", 300, 2368), ("w8a8", 3, 512), ("w8a8", 140, 512), ("w8a8", 100, 4032), ("fp4", 3, 512), ("fp4", 20, 512),
         ("fp4", 40, 512), ("fp4", 140, 512), ("fp4", 140, 2112)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("fmt,b,m", FORMS)
def test_slices(S, fmt, b, m, out):
    """y and residual as column slices of wider tensors, from odd columns; nothing else is written."""
    _say(f"slices {fmt} b={b} m={m} {out}")
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    n = 84
    c = Case(S, fmt, b, m, n, 16)
    for col, width in ((0, 96), (3, 101), (5, 92)):
        wide = torch.full((b, width), 77.0, dtype=dt, device="cuda")
        res = R.bf16(np.random.default_rng(col).standard_normal((b, n)))
        both = torch.zeros((b, 2 * n + 1), dtype=dt, device="cuda")  # residual and y beside each other
        both[:, :n] = dev(res.astype(np.float32), dt)
        y = c.call(c.qx, c.ascale, c.z, c.layer, act="silu", residual=both[:, :n], out_dtype=dt, y=wide[:, col:col + n])
        c.call(c.qx, c.ascale, c.z, c.layer, act="silu", residual=both[:, :n], out_dtype=dt, y=both[:, n + 1:])
        torch.cuda.synchronize()
        c.check(y, out, kind="silu", residual=res)
        c.check(both[:, n + 1:], out, kind="silu", residual=res)
        assert bool((both[:, n] == 0).all()) and np.array_equal(to_np(both[:, :n]), res)
        rest = torch.ones(width, dtype=torch.bool)
        rest[col:col + n] = False
        assert bool((wide[:, rest.cuda()] == 77.0).all())


@pytest.mark.parametrize("fmt,b,m", FORMS)
def test_unaligned_operands(S, fmt, b, m):
    """wscale, l2, bias, ascale and z at the least alignment that the header asks for."""
    _say(f"unaligned {fmt} b={b} m={m}")
    c = Case(S, fmt, b, m, 132, 24)

    def shifted(t):
        by = 2 if t.dtype == torch.uint8 else 1  # block scales: 2 bytes, others: one element
        w = torch.zeros(t.numel() + by, dtype=t.dtype, device="cuda")
        w[by:] = t.reshape(-1)
        return w[by:].view(t.shape)

    L = c.layer
    head = (L.m, L.n, L.rank) + ((L.t_x, L.t_w) if fmt == "fp4" else ())
    c.layer = type(L).from_tensors(*head, L.qw, shifted(L.wscale), None, shifted(L.l2), None, shifted(L.bias))
    c.ascale, c.z = shifted(c.ascale), shifted(c.z)
    c.run(act="silu", residual=True, gate_rows=b)


@pytest.mark.parametrize("fmt,b,m", FORMS + [("int4", 3, 512), ("int4", 140, 512)])
def test_nonfinite_rows_and_columns_stay_their_own(S, fmt, b, m):
    """NaN in a row's scale or z, infinity in another's z, NaN in a column's scale: the other outputs are as they were."""
    _say(f"nonfinite {fmt} b={b} m={m}")
    n = 70
    c = Case(S, fmt, b, m, n, 16)
    nan = 0x7F if fmt == "fp4" else float("nan")  # E4M3's NaN
    if fmt == "w8a8":
        c.ascale[0] = nan
        c.layer.wscale[9] = nan
    else:
        c.ascale[m // 64 - 1, 0] = nan
        c.layer.wscale[0, 9] = nan
    c.z[1, 3] = float("inf")
    if b > 3:
        c.z[b - 1, 0] = float("nan")
    rows = np.ones(b, bool)
    rows[[0, 1] + ([b - 1] if b > 3 else [])] = False
    cols = np.arange(n) != 9
    for act in ACTS:
        y = c.call(c.qx, c.ascale, c.z, c.layer, act=act, out_dtype=torch.float32)
        torch.cuda.synchronize()
        y = to_np(y)
        assert np.isnan(y[0]).all() and np.isnan(y[:, 9]).all(), act
        assert b <= 3 or np.isnan(y[b - 1]).all(), act
        assert act != "none" or not np.isfinite(y[1]).any()
        want, tol = R.epilogue(c.v[rows], c.dv[rows], act)
        assert (np.abs(y[rows] - want) <= tol)[:, cols].all(), act


@pytest.mark.parametrize("rows", [16, 32, 64])
@pytest.mark.parametrize("block", range(4))
def test_every_block_scale_in_the_row_kernel(S, block, rows):
    """NVFP4: each finite E4M3 scale of a row against every one of a column, `rows` rows a call."""
    _say(f"block scales {block} rows={rows}")
    rng = np.random.default_rng([block, rows])
    k = np.arange(127)
    e4m3 = np.where(k < 8, k / 8 * 2.0 ** -6, (1 + (k & 7) / 8) * 2.0 ** ((k >> 3) - 7.0))
    px, pw = np.zeros((127, 64), np.int64), rng.integers(0, 16, (127, 64))
    s = slice(16 * block, 16 * block + 16)
    px[:, s] = rng.integers(0, 16, (127, 16))
    ex, ew = rng.integers(0, 127, (127, 4)), rng.integers(0, 127, (127, 4))
    ex[:, block], ew[:, block] = k, rng.permutation(127)
    value = lambda p: E2M1[p & 7] * np.where(p & 8, -1, 1)
    x, w = value(px[:, s]) * e4m3[ex[:, block], None], value(pw[:, s]) * e4m3[ew[:, block], None]
    want, tol = R.epilogue(*R.product_values(x, w, 64))
    u8 = lambda t: torch.from_numpy(t).cuda()
    layer = S.DeviceLayerFp4.from_tensors(64, 127, 0, 1.0, 1.0, u8(LY.pack_fp4_codes(pw)), u8(LY.pack_fp4_scales(ew)))
    for lo in range(0, 127, rows):
        at = slice(lo, min(lo + rows, 127))
        y = S.svdq_fp4_gemm_lowrank_up_epi(u8(LY.pack_fp4_codes(px[at])), u8(LY.pack_fp4_scales(ex[at])), None, layer,
                                           out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert (np.abs(to_np(y) - want[at]) <= tol[at]).all(), lo


@pytest.mark.parametrize("rank", [0, 33])
@pytest.mark.parametrize("b,m,n", [(65, 1024, 64), (70, 4096, 1), (128, 1024, 129)])
def test_fp4_pieces_of_the_fewest_rows(S, b, m, n, rank):
    """Just past the row kernel: one or two tiles in two pieces and more."""
    _say(f"fp4 pieces b={b} m={m} n={n} rank={rank}")
    c = Case(S, "fp4", b, m, n, rank)
    c.run(out="f32")
    c.run(act="gelu_erf", act_begin=n // 3, gate_rows=7, residual=True, inplace=True, out="bf16")


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


def _whole_layer(S, fmt, m, n, rank, seed):
    """(layer, its linear call) with random codes, smoothing and branch."""
    c = Case(S, fmt, 1, m, n, rank, seed=seed)
    rng = np.random.default_rng([seed, m])
    l1 = torch.from_numpy(rng.standard_normal((rank, m)).astype(np.float32) / np.float32(np.sqrt(m))).cuda().bfloat16()
    inv = torch.from_numpy(np.exp(0.3 * rng.standard_normal(m)).astype(np.float32)).cuda()
    L = c.layer
    head = (m, n, rank) + ((L.t_x, L.t_w) if fmt == "fp4" else ())
    linear = {"int4": S.svdq_linear_epi, "w8a8": S.svdq_w8a8_linear_epi, "fp4": S.svdq_fp4_linear_epi}[fmt]
    return type(L).from_tensors(*head, L.qw, L.wscale, l1, L.l2, inv, L.bias), linear


@pytest.mark.parametrize("fmt", ["int4", "w8a8", "fp4"])
@pytest.mark.parametrize("b", [5, 150])
def test_whole_layers_in_a_graph(S, fmt, b):
    """Two layers one after the other in one graph, without workspaces of the caller's: replays equal eager calls."""
    _say(f"graph of whole layers {fmt} b={b}")
    m, n = 512, 2112
    (up, call), (down, _) = _whole_layer(S, fmt, m, n, 16, 1), _whole_layer(S, fmt, n, m, 24, 2)
    x = torch.randn(b, m, device="cuda").bfloat16()
    gate = torch.randn(1, m, device="cuda").bfloat16()
    y = torch.empty_like(x)

    def block(out):
        h = call(x, up, act="gelu_erf", act_begin=100)
        return call(h, down, gate=gate, residual=x, y=out)

    block(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block(y)
    for k in range(4):
        x.copy_(torch.randn_like(x))
        want = block(None)
        torch.cuda.synchronize()
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), k


@pytest.mark.parametrize("fmt", ["int4", "w8a8", "fp4"])
@pytest.mark.parametrize("b", [1, 40, 300])
def test_layer_in_place_on_its_input(S, fmt, b):
    """x is the residual and y too: the activations are quantized before the product writes."""
    _say(f"in place {fmt} b={b}")
    layer, call = _whole_layer(S, fmt, 1024, 1024, 16, 3)
    x = torch.randn(b, 1024, device="cuda").bfloat16()
    want = call(x, layer, act="silu", residual=x)
    got = call(x, layer, act="silu", residual=x, y=x)
    torch.cuda.synchronize()
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
