"""The products with an epilogue (activation, gate, residual) on the GPU against
64-bit references, in the INT4, 8-bit and NVFP4 settings.  Tolerances are the
error bounds of tests/epi_ref.py, element by element."""
import sys

import numpy as np
import pytest

from tests import epi_ref as R
from tests import layout as LY

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


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


def dev(v, dt):
    if dt == torch.bfloat16:
        return dev_bf16(v)
    return torch.from_numpy(np.ascontiguousarray(v)).cuda().to(dt)


def to_np(y):
    return y.float().cpu().numpy().astype(np.float64)


def scales(rng, shape, around):
    return (around * np.exp(0.4 * rng.standard_normal(shape))).astype(np.float16).astype(np.float64)


class Case:
    """One product's inputs, on the host in 64 bits and on the device."""

    def __init__(self, S, fmt, b, m, n, rank, bias=True, seed=0):
        rng = np.random.default_rng([seed, b, m, n, rank])
        self.S, self.fmt, self.b, self.n = S, fmt, b, n
        G = m // 64
        z = rng.standard_normal((b, rank)).astype(np.float32)
        l2 = R.bf16(0.3 * rng.standard_normal((n, rank)))
        bv = R.bf16(0.5 * rng.standard_normal(n)) if bias else None
        self.z = torch.from_numpy(z).cuda() if rank else None
        tl2 = dev_bf16(l2) if rank else None
        tb = dev_bf16(bv) if bias else None
        f16 = lambda v: torch.from_numpy(v.astype(np.float16)).cuda()
        if fmt == "int4":
            cx, cw = rng.integers(-7, 8, (b, m)), rng.integers(-7, 8, (n, m))
            sx, sw = scales(rng, (G, b), 0.2), scales(rng, (G, n), 0.05 / np.sqrt(m / 64))
            self.v, self.dv = R.product_int4(cx, sx, cw, sw, z, l2, bv)
            self.qx, self.ascale = torch.from_numpy(LY.pack_codes(cx)).cuda(), f16(sx)
            self.layer = S.DeviceLayer.from_tensors(m, n, rank, torch.from_numpy(LY.pack_codes(cw)).cuda(), f16(sw), None,
                                                    tl2, None, tb)
            self.call = S.svdq_gemm_w4a4_lowrank_up_epi
        elif fmt == "w8a8":
            cx, cw = rng.integers(-127, 128, (b, m)), rng.integers(-127, 128, (n, m))
            sx, sw = scales(rng, b, 0.01), scales(rng, n, 0.003 / np.sqrt(m / 64))
            # the integer sum is exact; conversion and scaling round once each
            v = (cx.astype(np.float64) @ cw.T.astype(np.float64)) * np.outer(sx, sw)
            self.v, self.dv = R._branch(v, np.abs(v), 2, z, l2, bv)
            self.qx, self.ascale = torch.from_numpy(LY.pack_codes8(cx)).cuda(), f16(sx)
            self.layer = S.DeviceLayer8.from_tensors(m, n, rank, torch.from_numpy(LY.pack_codes8(cw)).cuda(), f16(sw), None,
                                                     tl2, None, tb)
            self.call = S.svdq_w8a8_gemm_lowrank_up_epi
        else:
            px, pw = rng.integers(0, 16, (b, m)), rng.integers(0, 16, (n, m))
            ex, ew = rng.integers(40, 72, (b, m // 16)), rng.integers(40, 72, (n, m // 16))
            value = lambda p: E2M1[p & 7] * np.where(p & 8, -1, 1)
            e4m3 = lambda e: (1 + (e & 7) / 8) * 2.0 ** ((e >> 3) - 7.0)
            t_x, t_w = 2.0 ** -3, 2.0 ** -7
            x = value(px) * np.repeat(e4m3(ex), 16, 1) * t_x
            w = value(pw) * np.repeat(e4m3(ew), 16, 1) * t_w
            self.v, self.dv = R.product_values(x, w, m, z, l2, bv)  # an fp32 addition per channel
            u8 = lambda v: torch.from_numpy(v).cuda()
            self.qx, self.ascale = u8(LY.pack_fp4_codes(px)), u8(LY.pack_fp4_scales(ex))
            self.layer = S.DeviceLayerFp4.from_tensors(m, n, rank, t_x, t_w, u8(LY.pack_fp4_codes(pw)),
                                                       u8(LY.pack_fp4_scales(ew)), None, tl2, None, tb)
            self.call = S.svdq_fp4_gemm_lowrank_up_epi
        self.rng = rng

    def check(self, y, out, **epi):
        want, tol = R.epilogue(self.v, self.dv, out=out, **epi)
        err = np.abs(to_np(y) - want)
        bad = ~(err <= tol)
        assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, worst {np.max(err / tol):.3g} times the bound"

    def run(self, act="none", act_begin=0, gate_rows=None, residual=False, out="f32", inplace=False):
        dt = torch.bfloat16 if out == "bf16" else torch.float32
        gate = res = tg = tr = y = None
        if gate_rows is not None:
            gate = R.bf16(self.rng.standard_normal((-(-self.b // gate_rows), self.n)))
            tg = dev_bf16(gate)
        if residual:
            res = R.bf16(self.rng.standard_normal((self.b, self.n)))
            tr = dev(res.astype(np.float32), dt)
            y = tr if inplace else None
        y = self.call(self.qx, self.ascale, self.z, self.layer, act=act, act_begin=act_begin, gate=tg, gate_rows=gate_rows,
                      residual=tr, out_dtype=dt, y=y)
        torch.cuda.synchronize()
        self.check(y, out, kind=act, act_begin=act_begin, gate=gate, gate_rows=gate_rows, residual=res)


ACTS = ["none", "gelu_tanh", "gelu_erf", "silu", "relu"]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("fmt,b", [("int4", 3), ("int4", 150), ("w8a8", 150), ("fp4", 150)])
def test_activations(S, fmt, b, act):
    _say(f"act {fmt} b={b} {act}")
    c = Case(S, fmt, b, 256, 200, 16)
    for out in ("f32", "bf16"):
        c.run(act=act, out=out)
        c.run(act=act, act_begin=67, gate_rows=2 if b == 3 else 60, residual=True, out=out)


# rows: the row kernel's block sizes and their borders, one narrow tile, a tile border, split tiles (m = 2368 and
# 4096 at a few hundred rows), narrow tiles that would not pay as pieces (200 rows), whole wide tiles (1100 rows)
@pytest.mark.parametrize("b,m,n,rank", [
    (1, 64, 1, 0), (1, 4608, 77, 32), (2, 128, 16, 1), (15, 192, 33, 7), (16, 1024, 256, 16), (17, 2048, 61, 33),
    (32, 512, 130, 64), (33, 576, 18, 100), (64, 2048, 100, 256), (65, 64, 5, 8), (129, 1152, 260, 32), (256, 4096, 256, 16),
    (300, 2368, 203, 24), (4608, 640, 129, 8), (200, 1152, 4608, 16), (1100, 64, 5640, 40)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_int4_shapes(S, b, m, n, rank, out):
    _say(f"int4 b={b} m={m} n={n} rank={rank} {out}")
    c = Case(S, "int4", b, m, n, rank, bias=n % 2 == 0)
    c.run(out=out)
    c.run(act="gelu_tanh", act_begin=n // 3, gate_rows=max(1, b // 2), residual=True, out=out, inplace=True)


@pytest.mark.parametrize("fmt", ["w8a8", "fp4"])
# 8-bit: 64 x 64 tiles up to 384 wide ones, split tiles where those are few and long, whole wide tiles (the last)
@pytest.mark.parametrize("b,m,n,rank", [(1, 64, 1, 0), (5, 192, 70, 9), (256, 4096, 256, 16), (300, 2368, 201, 33),
                                        (300, 4352, 130, 40), (1100, 64, 5640, 20)])
def test_other_settings_shapes(S, fmt, b, m, n, rank):
    _say(f"{fmt} b={b} m={m} n={n} rank={rank}")
    c = Case(S, fmt, b, m, n, rank, bias=n % 2 == 0)
    for out in ("f32", "bf16"):
        c.run(out=out)
        c.run(act="silu", act_begin=n // 2, gate_rows=max(1, b // 3), residual=True, out=out, inplace=True)


def test_split_tail_behind_full_rounds(S):
    """Whole tiles and split tiles in one launch (epilogue in the kernel and in the reduction)."""
    b, m, n = 4608, 1536, 2944
    info = S.svdq_gemm_schedule(b, n, m)
    _say(f"schedule {info}")
    assert 0 < info["split_tiles"] < info["tiles"]
    c = Case(S, "int4", b, m, n, 16)
    c.run(act="gelu_tanh", act_begin=1000, gate_rows=1000, residual=True, out="bf16")


@pytest.mark.parametrize("b", [3, 40, 140])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_slices_and_alignment(S, b, out):
    """y and residual as column slices of wider tensors, from odd columns; nothing else is written."""
    _say(f"slices b={b} {out}")
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    n = 84
    c = Case(S, "int4", b, 512, n, 16)
    for col, width in ((0, 96), (4, 100), (3, 101), (5, 92)):
        wide = torch.full((b, width), 77.0, dtype=dt, device="cuda")
        res = R.bf16(np.random.default_rng(col).standard_normal((b, n)))
        both = torch.zeros((b, 2 * n + 1), dtype=dt, device="cuda")  # residual and y beside each other
        both[:, :n] = dev(res.astype(np.float32), dt)
        y = c.call(c.qx, c.ascale, c.z, c.layer, act="relu", residual=both[:, :n], out_dtype=dt, y=wide[:, col:col + n])
        c.call(c.qx, c.ascale, c.z, c.layer, act="relu", residual=both[:, :n], out_dtype=dt, y=both[:, n + 1:])
        torch.cuda.synchronize()
        c.check(y, out, kind="relu", residual=res)
        c.check(both[:, n + 1:], out, kind="relu", residual=res)
        assert bool((both[:, n] == 0).all()) and np.array_equal(to_np(both[:, :n]), res)
        rest = torch.ones(width, dtype=torch.bool)
        rest[col:col + n] = False
        assert bool((wide[:, rest.cuda()] == 77.0).all())


@pytest.mark.parametrize("b", [1, 20, 200])
def test_unaligned_scales_and_factors(S, b):
    """wscale, l2, bias, ascale and z at element alignment only."""
    _say(f"unaligned b={b}")
    c = Case(S, "int4", b, 512, 132, 24)

    def shifted(t):
        w = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        w[1:] = t.reshape(-1)
        return w[1:].view(t.shape)

    L = c.layer
    c.layer = S.DeviceLayer.from_tensors(L.m, L.n, L.rank, L.qw, shifted(L.wscale), None, shifted(L.l2), None,
                                         shifted(L.bias))
    c.ascale, c.z = shifted(c.ascale), shifted(c.z)
    c.run(act="silu", residual=True, gate_rows=b)


@pytest.mark.parametrize("b", [5, 100])
def test_nonfinite_rows_stay_their_own(S, b):
    """A row with NaN or infinite scales, z or residual leaves the other rows as they are; activations of large and
    infinite values."""
    _say(f"nonfinite b={b}")
    c = Case(S, "int4", b, 256, 70, 16)
    c.ascale[0, 0] = float("nan")
    c.ascale[1, 1] = float("inf")
    c.z[2, 0] = float("nan")
    for act in ACTS:
        y = c.call(c.qx, c.ascale, c.z, c.layer, act=act, out_dtype=torch.float32)
        torch.cuda.synchronize()
        y = to_np(y)
        assert np.isnan(y[0]).all() and np.isnan(y[2]).all(), act
        assert not np.isfinite(y[1]).any() or act != "none"
        want, tol = R.epilogue(c.v[3:], c.dv[3:], act)
        assert (np.abs(y[3:] - want) <= tol).all(), act


def test_activation_extremes(S):
    """v through the bias alone: large magnitudes, both signs, zeros, infinities, NaN."""
    vals = np.array([0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 4.0, -4.0, 9.5, -9.5, 30.0, -30.0, 100.0, -100.0, 1e10, -1e10,
                     3e38, -3e38, np.inf, np.nan])
    n = len(vals)
    for b in (2, 130):
        _say(f"extremes b={b}")
        qx = torch.zeros((1, b, 32), dtype=torch.uint8, device="cuda")
        asc = torch.zeros((1, b), dtype=torch.float16, device="cuda")
        layer = S.DeviceLayer.from_tensors(64, n, 0, torch.zeros((1, n, 32), dtype=torch.uint8, device="cuda"),
                                           torch.zeros((1, n), dtype=torch.float16, device="cuda"), None, None, None,
                                           torch.tensor(vals, dtype=torch.float32).bfloat16().cuda())
        v = torch.tensor(vals, dtype=torch.float32).bfloat16().double().numpy()
        for act in ACTS:
            y = to_np(S.svdq_gemm_w4a4_lowrank_up_epi(qx, asc, None, layer, act=act, out_dtype=torch.float32))
            assert np.isnan(y[:, -1]).all() and (y[:, -2] == np.inf).all(), act
            want, tol = R.epilogue(v[None, :-2], np.zeros((1, n - 2)), act)
            assert (np.abs(y[:, :-2] - want) <= tol).all(), (act, np.abs(y[:, :-2] - want).max(0))


def test_same_inputs_same_bits_and_side_stream(S):
    for b in (4, 300):
        c = Case(S, "int4", b, 2368, 203, 24)
        args = dict(act="gelu_erf", act_begin=5, out_dtype=torch.float32)
        y0 = c.call(c.qx, c.ascale, c.z, c.layer, **args)
        y1 = c.call(c.qx, c.ascale, c.z, c.layer, **args)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y2 = c.call(c.qx, c.ascale, c.z, c.layer, stream=side, **args)
        y3 = c.call(c.qx, c.ascale, c.z, c.layer, stream=side.cuda_stream, **args)
        torch.cuda.synchronize()
        for y in (y1, y2, y3):
            assert torch.equal(y, y0)


def test_b0(S):
    c = Case(S, "int4", 1, 64, 20, 4)
    qx, asc = torch.empty((1, 0, 32), dtype=torch.uint8, device="cuda"), torch.empty((1, 0), dtype=torch.float16, device="cuda")
    z = torch.empty((0, 4), device="cuda")
    assert S.svdq_gemm_w4a4_lowrank_up_epi(qx, asc, z, c.layer, act="silu").shape == (0, 20)


@pytest.mark.parametrize("fmt", ["int4", "w8a8", "fp4"])
@pytest.mark.parametrize("b", [1, 7, 200])
def test_whole_layer_is_its_two_steps(S, fmt, b):
    """svdq_*linear_epi equals, bit for bit, quantization and product called one after the other."""
    from oracle import svdq_oracle as O
    _say(f"linear_epi {fmt} b={b}")
    m, n, rank = 512, 132, 16
    rng = np.random.default_rng(b)
    xb = LY.f32_to_bf16_bits(R.bf16(rng.standard_normal((b, m))).astype(np.float32))
    w = (rng.standard_normal((m, n)) / np.sqrt(m)).astype(np.float32)
    a = O.act_amax(LY.bf16_bits_to_f32(xb))
    x = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.bfloat16)
    bias = LY.f32_to_bf16_bits(R.bf16(rng.standard_normal(n)).astype(np.float32))
    res = torch.randn(b, n, device="cuda").bfloat16()
    gate = torch.randn(1, n, device="cuda").bfloat16()
    epi = dict(act="gelu_tanh", act_begin=40, gate=gate, residual=res)
    if fmt == "int4":
        L = S.DeviceLayer(LY.oracle_layer_to_host_abi(O.prepare_weights(w, a, rank)), bias=bias)
        q = S.svdq_quantize_act_lowrank_down(x, L.smooth_inv, L.l1, rank)
        y, want = S.svdq_linear_epi(x, L, **epi), S.svdq_gemm_w4a4_lowrank_up_epi(*q, L, **epi)
    elif fmt == "w8a8":
        L = S.DeviceLayer8(LY.oracle_w8a8_to_host_abi(O.prepare_weights_w8a8(w, a, rank)), bias=bias)
        q = S.svdq_w8a8_quantize_act_lowrank_down(x, L.smooth_inv, L.l1, rank)
        y, want = S.svdq_w8a8_linear_epi(x, L, **epi), S.svdq_w8a8_gemm_lowrank_up_epi(*q, L, **epi)
    else:
        L = S.DeviceLayerFp4(LY.oracle_fp4_to_host_abi(O.prepare_weights_fp4(w, a, rank), O.e4m3_bits), bias=bias)
        q = S.svdq_fp4_quantize_act_lowrank_down(x, L.smooth_inv, L.l1, rank, L.t_x)
        y, want = S.svdq_fp4_linear_epi(x, L, **epi), S.svdq_fp4_gemm_lowrank_up_epi(*q, L, **epi)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("b", [4, 300])
def test_graph_replay(S, b):
    """Replays on new inputs, with eager calls between them, equal the eager result."""
    _say(f"graph b={b}")
    c = Case(S, "int4", b, 2368, 203, 24)
    y = torch.zeros(b, 203, device="cuda")
    res = torch.randn(b, 203, device="cuda")
    ws = torch.empty(max(1, S.svdq_gemm_epi_workspace_size(b, 203, 2368)), dtype=torch.uint8, device="cuda")
    call = lambda out, w: c.call(c.qx, c.ascale, c.z, c.layer, act="silu", residual=res, out_dtype=torch.float32, y=out,
                                 workspace=w)
    call(y, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y, ws)
    for k in range(3):
        c.z.copy_(torch.randn_like(c.z))
        res.copy_(torch.randn_like(res))
        want = call(None, None)
        torch.cuda.synchronize()
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), k


@pytest.mark.parametrize("seed", range(24))
def test_random_products(S, seed):
    rng = np.random.default_rng([7, seed])
    fmt = ["int4", "int4", "w8a8", "fp4"][rng.integers(4)]
    b, n = int(np.exp(rng.uniform(0, np.log(700)))), int(np.exp(rng.uniform(0, np.log(900))))
    m, rank = 64 * int(rng.integers(1, 40)), int(rng.choice([0, 1, 8, 20, 32, 50, 64, 129]))
    kw = dict(act=ACTS[rng.integers(5)], act_begin=int(rng.integers(0, n + 1)), residual=bool(rng.integers(2)),
              gate_rows=[None, int(rng.integers(1, b + 1))][rng.integers(2)], out=["f32", "bf16"][rng.integers(2)],
              inplace=bool(rng.integers(2)))
    _say(f"random {fmt} b={b} m={m} n={n} rank={rank} {kw}")
    Case(S, fmt, b, m, n, rank, bias=bool(rng.integers(2)), seed=seed).run(**kw)


def test_outputs_past_32_bit_offsets(S):
    """More than 2^31 outputs: the first and last rows, in place on the residual."""
    b, m, n = 66000, 64, 33000
    rng = np.random.default_rng(3)
    rows = np.array([0, 1, 127, 128, 65071, 65073, 65535, 65536, b - 129, b - 1])
    cx, cw = np.zeros((b, m), np.int8), rng.integers(-7, 8, (n, m)).astype(np.int8)
    cx[rows] = rng.integers(-7, 8, (len(rows), m))
    sx, sw = np.full((1, b), 0.25), (0.05 * np.exp(0.4 * rng.standard_normal((1, n)))).astype(np.float16).astype(np.float64)
    layer = S.DeviceLayer.from_tensors(m, n, 0, torch.from_numpy(LY.pack_codes(cw)).cuda(),
                                       torch.from_numpy(sw.astype(np.float16)).cuda())
    y = torch.full((b, n), 1.5, dtype=torch.bfloat16, device="cuda")
    assert y.numel() > 2 ** 31
    S.svdq_gemm_w4a4_lowrank_up_epi(torch.from_numpy(LY.pack_codes(cx)).cuda(), torch.from_numpy(sx.astype(np.float16)).cuda(),
                                    None, layer, act="silu", act_begin=100, residual=y, y=y)
    torch.cuda.synchronize()
    got = to_np(y[torch.from_numpy(rows).cuda()])
    v, dv = R.product_int4(cx[rows], sx[:, rows], cw, sw)
    want, tol = R.epilogue(v, dv, "silu", 100, residual=np.full(v.shape, 1.5), out="bf16")
    assert (np.abs(got - want) <= tol).all()
    assert bool((y[2:127] == 1.5).all()) and bool((y[65537:65600] == 1.5).all())
    # the same rows combined: the index reaches past 2^31 elements
    out = S.svdq_combine_rows(y, torch.tensor([[0, b - 1]], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    both = got[0] + got[-1]
    assert (np.abs(to_np(out)[0] - both) <= np.abs(both) * 2.0 ** -8 + 1e-30).all()


@pytest.mark.parametrize("block", range(4))
def test_every_block_scale(S, block):
    """NVFP4: each finite E4M3 scale against each other, one block of the group at a time."""
    rng = np.random.default_rng(block)
    k = np.arange(127)
    e4m3 = np.where(k < 8, k / 8 * 2.0 ** -6, (1 + (k & 7) / 8) * 2.0 ** ((k >> 3) - 7.0))
    px, pw = np.zeros((127, 64), np.int64), rng.integers(0, 16, (127, 64))
    s = slice(16 * block, 16 * block + 16)
    px[:, s] = rng.integers(0, 16, (127, 16))
    ex, ew = rng.integers(0, 127, (127, 4)), rng.integers(0, 127, (127, 4))
    ex[:, block], ew[:, block] = k, rng.permutation(127)
    value = lambda p: E2M1[p & 7] * np.where(p & 8, -1, 1)
    x, w = value(px[:, s]) * e4m3[ex[:, block], None], value(pw[:, s]) * e4m3[ew[:, block], None]
    v, dv = R.product_values(x, w, 64)
    u8 = lambda t: torch.from_numpy(t).cuda()
    layer = S.DeviceLayerFp4.from_tensors(64, 127, 0, 1.0, 1.0, u8(LY.pack_fp4_codes(pw)), u8(LY.pack_fp4_scales(ew)))
    y = S.svdq_fp4_gemm_lowrank_up_epi(u8(LY.pack_fp4_codes(px)), u8(LY.pack_fp4_scales(ex)), None, layer,
                                       out_dtype=torch.float32)
    torch.cuda.synchronize()
    want, tol = R.epilogue(v, dv)
    assert (np.abs(to_np(y) - want) <= tol).all()


@pytest.mark.parametrize("rank", [0, 33])
@pytest.mark.parametrize("b,m,n", [(1, 1024, 64), (130, 2112, 301), (256, 1088, 1000), (100, 8192, 130)])
def test_fp4_pieces(S, b, m, n, rank):
    """Few tiles, which are split over the channel groups: every part of the epilogue after the sum of the pieces."""
    case = Case(S, "fp4", b, m, n, rank)
    case.run(out="f32")
    case.run(act="gelu_erf", act_begin=n // 3, gate_rows=7, residual=True, inplace=True, out="bf16")


@pytest.mark.parametrize("rank", [0, 5, 40])
@pytest.mark.parametrize("b,m,n", [(1, 64, 1), (1, 4608, 70), (15, 192, 33), (17, 1152, 130), (33, 448, 999), (64, 2048, 50)])
def test_fp4_few_rows(S, b, m, n, rank):
    case = Case(S, "fp4", b, m, n, rank, bias=rank != 5)
    case.run(out="f32")
    case.run(act="silu", act_begin=n // 2, gate_rows=4, residual=True, inplace=True, out="bf16")


@pytest.mark.parametrize("b", [7, 130])
def test_fp4_in_two_graphs_and_on_two_streams(S, b):
    """Captured calls (row kernel, split tiles) of two layers, replayed together on two streams, each with its workspace."""
    n, m = 203, 2368
    runs = []
    for seed in range(2):
        c = Case(S, "fp4", b, m, n, 24, seed=seed)
        y = torch.empty((b, n), device="cuda")
        ws = torch.empty(max(1, S.svdq_fp4_gemm_workspace_size(b, n, m)), dtype=torch.uint8, device="cuda")
        call = lambda c=c, y=y, ws=ws: c.call(c.qx, c.ascale, c.z, c.layer, act="gelu_tanh", out_dtype=torch.float32, y=y,
                                              workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((c, y, g, torch.cuda.Stream()))
    for k in range(3):
        for c, y, g, stream in runs:
            y.zero_()
            c.z.copy_(torch.randn_like(c.z))
        torch.cuda.synchronize()
        for c, y, g, stream in runs:
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for c, y, g, stream in runs:
            want = c.call(c.qx, c.ascale, c.z, c.layer, act="gelu_tanh", out_dtype=torch.float32)
            torch.cuda.synchronize()
            assert torch.equal(y, want), (k, b)
