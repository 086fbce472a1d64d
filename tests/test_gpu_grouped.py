"""INT4 layers grouped by expert, and the combination of their rows, on the GPU
against 64-bit references (tests/epi_ref.py gives the error bounds)."""
import sys

import numpy as np
import pytest

from tests import epi_ref as R
from tests import layout as LY

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


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


class Experts:
    """E random layers on the host in 64 bits and stacked on the device."""

    def __init__(self, S, E, m, n, rank, bias=True, smooth=True, seed=0):
        rng = np.random.default_rng([seed, E, m, n, rank])
        G = m // 64
        self.E, self.m, self.n, self.rank = E, m, n, rank
        self.cw = rng.integers(-7, 8, (E, n, m)).astype(np.int8)
        self.sw = (0.05 / np.sqrt(G) * np.exp(0.4 * rng.standard_normal((E, G, n)))).astype(np.float16).astype(np.float64)
        self.l1 = R.bf16(rng.standard_normal((E, rank, m)) / np.sqrt(m))
        self.l2 = R.bf16(0.3 * rng.standard_normal((E, n, rank)))
        self.bias = R.bf16(0.5 * rng.standard_normal((E, n))) if bias else None
        self.inv = np.exp(0.5 * rng.standard_normal((E, m))).astype(np.float32) if smooth else None
        self.layer = S.GroupedDeviceLayer.from_tensors(
            E, m, n, rank, torch.from_numpy(np.stack([LY.pack_codes(c) for c in self.cw])).cuda(),
            torch.from_numpy(self.sw.astype(np.float16)).cuda(), dev_bf16(self.l1) if rank else None,
            dev_bf16(self.l2) if rank else None, torch.from_numpy(self.inv).cuda() if smooth else None,
            dev_bf16(self.bias) if bias else None)

    def quantized(self, e, x):
        """(codes, scales, z, dz) of rows x of expert e."""
        xt, q, s = R.quantize(x, self.inv[e] if self.inv is not None else None)
        z, a = xt @ self.l1[e].T, np.abs(xt) @ np.abs(self.l1[e]).T
        return q, s, z, (self.m + 24) * 2 * R.U * a


def unpack(qx, rows):
    return LY.unpack_codes(qx.cpu().numpy())[rows]


def check_quantized(X, x, off, src, qx, ascale, z, sentinel):
    codes = LY.unpack_codes(qx.cpu().numpy())
    asc = ascale.cpu().numpy().astype(np.float64)
    zz = None if z is None else to_np(z)
    live = np.zeros(len(src), bool)
    for e in range(X.E):
        lo, hi = off[e], off[e + 1]
        live[lo:hi] = True
        rows = np.where((src[lo:hi] >= 0)[:, None] & (src[lo:hi] < len(x))[:, None], x[np.clip(src[lo:hi], 0, len(x) - 1)], 0)
        q, s, zr, dz = X.quantized(e, rows)
        assert np.array_equal(codes[lo:hi], q), e
        assert np.array_equal(asc[:, lo:hi], s), e
        if zz is not None:
            assert (np.abs(zz[lo:hi] - zr) <= dz + 1e-38).all(), e
    # rows without an expert keep what was there
    assert (qx.cpu().numpy()[:, ~live] == sentinel).all()
    if zz is not None:
        assert (zz[~live] == sentinel).all()


def ragged(rng, E, b, empty=0.3, pad=0):
    w = rng.random(E) * (rng.random(E) > empty) + 1e-9
    cuts = np.sort(rng.choice(b - pad + 1, E - 1)) if E > 1 else np.zeros(0, int)
    c = np.diff(np.concatenate([[0], cuts, [b - pad]]))
    if w.max() > 1e-9 and E > 1:  # some experts without rows
        for e in np.nonzero(w < 1e-8)[0]:
            c[(e + 1) % E] += c[e]
            c[e] = 0
    return np.concatenate([[0], np.cumsum(c)])


@pytest.mark.parametrize("E,b,m,rank,pad", [
    (1, 1, 64, 0, 0), (1, 17, 128, 16, 0), (3, 5, 192, 7, 0), (4, 70, 1024, 32, 9), (8, 200, 640, 48, 0), (5, 33, 256, 100, 3),
    (3, 40, 576, 256, 0), (64, 90, 128, 33, 5), (65, 300, 128, 64, 0), (130, 40, 64, 20, 1), (1024, 700, 64, 8, 0)])
@pytest.mark.parametrize("gather", [False, True])
def test_quantize(S, E, b, m, rank, pad, gather):
    _say(f"quantize E={E} b={b} m={m} rank={rank} pad={pad} gather={gather}")
    rng = np.random.default_rng([E, b, m])
    X = Experts(S, E, m, 16, rank, smooth=E != 3)
    off = ragged(rng, E, b, pad=pad)
    rows = 23 if gather else b
    x = R.bf16(rng.standard_normal((rows, m)) * np.exp(rng.standard_normal((rows, 1))))
    x[0] = 0
    x[rows // 2, :64] = 0
    src = rng.integers(0, rows, b) if gather else np.arange(b)
    if gather and b > 4:
        src[:4] = [-1, rows, 1 << 30, src[4]]  # rows that are not there, and one row twice
    G = m // 64
    qx = torch.full((G, b, 32), 99, dtype=torch.uint8, device="cuda")
    asc = torch.full((G, b), 99.0, dtype=torch.float16, device="cuda")
    z = torch.full((b, rank), 99.0, device="cuda") if rank else None
    S.svdq_grouped_quantize_act_lowrank_down(dev_bf16(x), i32(off), X.layer, i32(src) if gather else None, qx, asc, z)
    torch.cuda.synchronize()
    check_quantized(X, x, off, src, qx, asc, z, 99)


# the row kernel's block sizes, the 64-row tiles (many small experts; many channels), the 128-row tiles (the last two)
@pytest.mark.parametrize("E,b,m,n,rank,pad", [
    (1, 1, 64, 1, 0, 0), (2, 3, 4608, 40, 32, 0), (16, 9, 512, 77, 16, 2), (7, 100, 192, 33, 7, 0), (3, 80, 1024, 130, 33, 10),
    (4, 200, 256, 64, 100, 0), (64, 500, 128, 36, 16, 7), (100, 900, 64, 20, 3, 0), (1024, 700, 64, 40, 8, 3), (3, 400, 640, 203, 24, 11),
    (5, 1500, 192, 300, 0, 0), (2, 300, 2048, 129, 256, 1), (64, 1500, 64, 1100, 20, 3), (130, 1400, 128, 1283, 0, 0),
    (3, 400, 4096, 3000, 33, 11), (2, 1100, 128, 11001, 16, 5), (1, 1100, 64, 11264, 40, 0)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_product(S, E, b, m, n, rank, pad, out):
    _say(f"product E={E} b={b} m={m} n={n} rank={rank} pad={pad} {out}")
    rng = np.random.default_rng([E, b, m, n])
    X = Experts(S, E, m, n, rank, bias=n % 2 == 0)
    off = ragged(rng, E, b, pad=pad)
    G = m // 64
    cx = rng.integers(-7, 8, (b, m))
    sx = (0.2 * np.exp(0.4 * rng.standard_normal((G, b)))).astype(np.float16).astype(np.float64)
    z = rng.standard_normal((b, rank)).astype(np.float32)
    sd, zd = sx.copy(), z.copy()
    if pad:  # what lies behind the last expert's rows is not used
        sd[:, b - pad:] = np.nan
        zd[b - pad:] = np.nan
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    for act, begin, wide in (("none", 0, False), ("gelu_tanh", n // 3, True)):
        buf = torch.full((b, n + (5 if wide else 0)), 99.0, dtype=dt, device="cuda")
        y = buf[:, 2:2 + n] if wide else buf
        S.svdq_grouped_gemm_w4a4_lowrank_up(torch.from_numpy(LY.pack_codes(cx)).cuda(),
                                            torch.from_numpy(sd.astype(np.float16)).cuda(),
                                            torch.from_numpy(zd).cuda() if rank else None, i32(off), X.layer, act=act,
                                            act_begin=begin, out_dtype=dt, y=y)
        torch.cuda.synchronize()
        got = to_np(y)
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            v, dv = R.product_int4(cx[lo:hi], sx[:, lo:hi], X.cw[e], X.sw[e], z[lo:hi], X.l2[e],
                                   X.bias[e] if X.bias is not None else None)
            want, tol = R.epilogue(v, dv, act, begin, out=out)
            err = np.abs(got[lo:hi] - want)
            assert (err <= tol).all(), (e, act, np.max(err / tol))
        assert (got[off[-1]:] == 99).all()
        if wide:
            assert bool((buf[:, :2] == 99).all()) and bool((buf[:, 2 + n:] == 99).all())


@pytest.mark.parametrize("E,b,n", [(4, 6, 20), (4, 150, 36), (3, 900, 40)])
def test_offsets_of_any_content(S, E, b, n):
    """Rows before the first offset and behind the last keep their contents; offsets outside [0, b] are clamped;
    decreasing ones write no row but those between the smallest and the largest."""
    _say(f"offsets E={E} b={b} n={n}")
    m = 128
    X = Experts(S, E, m, n, 8)
    rng = np.random.default_rng(b)
    x = R.bf16(rng.standard_normal((b, m)))
    dx = dev_bf16(x)

    def run(off):
        y = torch.full((b, n), 99.0, device="cuda")
        S.svdq_grouped_linear(dx, i32(off), X.layer, y=y)
        torch.cuda.synchronize()
        return to_np(y)

    full = run([0] + [b // 2] * (E - 1) + [b])  # experts 0 and E-1 only
    assert (full != 99).all()
    same = run([-5] + [b // 2] * (E - 1) + [b + 1000])
    assert np.array_equal(full, same)
    part = run([2] + [b // 2] * (E - 1) + [b - 1])
    assert (part[:2] == 99).all() and (part[b - 1:] == 99).all()
    assert (run([b] * (E + 1)) == 99).all() and (run([0] * (E + 1)) == 99).all()
    assert (run([-(1 << 31)] * (E + 1)) == 99).all() and (run([(1 << 31) - 1] * (E + 1)) == 99).all()
    down = run([b - 1] + [b // 2] * (E - 1) + [1])
    assert (down == 99).all()
    saw = [1, b - 1] * (E + 1)
    got = run(saw[:E + 1])
    assert (got[:1] == 99).all() and (got[b - 1:] == 99).all()


@pytest.mark.parametrize("E,tokens,k,m,n,rank", [(6, 1, 2, 256, 100, 16), (8, 40, 3, 512, 72, 32), (5, 300, 2, 192, 130, 70)])
def test_linear_is_its_two_steps_and_right(S, E, tokens, k, m, n, rank):
    _say(f"linear E={E} tokens={tokens} k={k} m={m} n={n} rank={rank}")
    rng = np.random.default_rng(tokens)
    X = Experts(S, E, m, n, rank)
    x = R.bf16(rng.standard_normal((tokens, m)))
    chosen = np.stack([rng.choice(E, k, replace=False) for _ in range(tokens)]).reshape(-1)
    order = np.argsort(chosen, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(chosen, minlength=E))])
    src = order // k
    dx, do, ds = dev_bf16(x), i32(off), i32(src)
    y = S.svdq_grouped_linear(dx, do, X.layer, ds, act="silu", out_dtype=torch.float32)
    q = S.svdq_grouped_quantize_act_lowrank_down(dx, do, X.layer, ds)
    want = S.svdq_grouped_gemm_w4a4_lowrank_up(*q, do, X.layer, act="silu", out_dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = S.svdq_grouped_linear(dx, do, X.layer, ds, act="silu", out_dtype=torch.float32, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(y2, want)
    zz = to_np(q[2])
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        codes, s, _, _ = X.quantized(e, x[src[lo:hi]])
        v, dv = R.product_int4(codes, s, X.cw[e], X.sw[e], zz[lo:hi], X.l2[e], X.bias[e])
        ref, tol = R.epilogue(v, dv, "silu")
        assert (np.abs(to_np(y[lo:hi]) - ref) <= tol).all(), e


def test_matches_single_layers(S):
    """Each expert's rows agree with svdq_linear_epi on that expert's layer: codes and scales bit for bit, results
    within the two bounds."""
    E, m, n, rank, b = 3, 512, 96, 16, 60
    X = Experts(S, E, m, n, rank)
    rng = np.random.default_rng(1)
    x = R.bf16(rng.standard_normal((b, m)))
    off = np.array([0, 20, 20, 60])
    dx = dev_bf16(x)
    qx, asc, _ = S.svdq_grouped_quantize_act_lowrank_down(dx, i32(off), X.layer)
    L = X.layer
    for e in (0, 2):
        lo, hi = off[e], off[e + 1]
        one = S.DeviceLayer.from_tensors(m, n, rank, L.qw[e], L.wscale[e], L.l1[e], L.l2[e], L.smooth_inv[e], L.bias[e])
        q1, a1, _ = S.svdq_quantize_act_lowrank_down(dx[lo:hi].contiguous(), one.smooth_inv, one.l1, rank)
        assert torch.equal(qx[:, lo:hi], q1) and torch.equal(asc[:, lo:hi], a1)


def test_graph_replay_with_new_routing(S):
    E, m, n, rank, tokens, k = 6, 256, 100, 16, 50, 2
    X = Experts(S, E, m, n, rank)
    rng = np.random.default_rng(2)
    b = tokens * k
    x = torch.zeros(tokens, m, dtype=torch.bfloat16, device="cuda")
    off, src = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(b, dtype=torch.int32, device="cuda")
    index = torch.zeros(tokens, k, dtype=torch.int32, device="cuda")
    y, out = torch.zeros(b, n, device="cuda"), torch.zeros(tokens, n, device="cuda")
    ws = torch.empty(S.svdq_grouped_linear_workspace_size(b, E, m, n, rank), dtype=torch.uint8, device="cuda")

    def step(y, out, ws):
        S.svdq_grouped_linear(x, off, X.layer, src, act="gelu_tanh", out_dtype=torch.float32, y=y, workspace=ws)
        return S.svdq_combine_rows(y, index, residual=out, y=out)

    step(y, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(y, out, ws)
    for it in range(3):
        chosen = rng.integers(0, E if it else 1, b)
        order = np.argsort(chosen, kind="stable")
        off.copy_(i32(np.concatenate([[0], np.cumsum(np.bincount(chosen, minlength=E))])))
        src.copy_(i32(order // k))
        index.copy_(i32(np.argsort(order).reshape(tokens, k)))
        x.copy_(torch.randn(tokens, m, device="cuda"))
        start = torch.randn(tokens, n, device="cuda")
        want = step(torch.zeros_like(y), start.clone(), torch.empty_like(ws))
        torch.cuda.synchronize()
        y.zero_()
        out.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), it


@pytest.mark.parametrize("t,k,n,rows", [(1, 1, 1, 1), (3, 2, 8, 6), (7, 2, 77, 14), (40, 9, 264, 100), (5, 20, 1152, 30), (300, 6, 100, 1800)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_combine(S, t, k, n, rows, out):
    _say(f"combine t={t} k={k} n={n} rows={rows} {out}")
    rng = np.random.default_rng([t, k, n])
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    v = R.bf16(rng.standard_normal((rows, n))) if out == "bf16" else rng.standard_normal((rows, n)).astype(np.float32)
    res = R.bf16(rng.standard_normal((t, n)))
    idx = rng.integers(-1, rows + 1, (t, k))
    w = rng.standard_normal((t, k)).astype(np.float32)
    d = lambda a: dev_bf16(a) if dt == torch.bfloat16 else torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()
    ok = (idx >= 0) & (idx < rows)
    for weight, residual in ((w, res), (None, None), (w, None)):
        ww = np.where(ok, w if weight is not None else 1.0, 0.0).astype(np.float64)
        terms = ww[..., None] * v.astype(np.float64)[np.clip(idx, 0, rows - 1)]
        want, mag = terms.sum(1), np.abs(terms).sum(1)
        if residual is not None:
            want, mag = want + res, mag + np.abs(res)
        # k fused additions and the residual's, then the output's rounding
        tol = (k + 2) * R.U * mag * 1.01 + np.abs(want) * (2.0 ** -8 if out == "bf16" else R.U) * 1.01 + 1e-38
        tr = d(res) if residual is not None else None
        y = S.svdq_combine_rows(d(v), i32(idx), torch.from_numpy(w).cuda() if weight is not None else None, residual=tr)
        torch.cuda.synchronize()
        assert (np.abs(to_np(y) - want) <= tol).all()
        if tr is not None:  # in place
            y2 = S.svdq_combine_rows(d(v), i32(idx), torch.from_numpy(w).cuda(), residual=tr, y=tr)
            torch.cuda.synchronize()
            assert torch.equal(y2, y)


def test_combine_unaligned_and_missing_nan_rows(S):
    """A row that no index names may hold anything; pointers at element alignment."""
    for dt in (torch.bfloat16, torch.float32):
        base = torch.randn(1 + 10 * 16, device="cuda").to(dt)
        rows = base[1:].view(10, 16)
        rows[9] = float("nan")
        idx = i32([[0, 3], [8, -1], [10, 11]])
        y = S.svdq_combine_rows(rows, idx)
        torch.cuda.synchronize()
        f = rows.double()
        want = torch.stack([f[0] + f[3], f[8], f[8] * 0])
        assert bool(((y.double() - want).abs() <= want.abs() * (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -23)).all())


def test_a_whole_expert_block(S):
    """fc1 with its activation, fc2, and the weighted sum onto the residual stream, as a model chains them, against the
    same chain of dense 64-bit layers; the library's codes may fall on the other side of a rounding border where the
    32-bit activation differs, so the block is held to the layers' 4-bit step."""
    E, m, h, rank, tokens, k = 4, 256, 512, 16, 30, 2
    A, B = Experts(S, E, m, h, rank, seed=1), Experts(S, E, h, m, rank, seed=2)
    rng = np.random.default_rng(5)
    x = R.bf16(rng.standard_normal((tokens, m)))
    chosen = np.stack([rng.choice(E, k, replace=False) for _ in range(tokens)])
    flat = chosen.reshape(-1)
    order = np.argsort(flat, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    w = rng.random((tokens, k)).astype(np.float32)
    dx, do = dev_bf16(x), i32(off)
    mid = S.svdq_grouped_linear(dx, do, A.layer, i32(order // k), act="gelu_tanh")
    rows = S.svdq_grouped_linear(mid, do, B.layer)
    y = S.svdq_combine_rows(rows, i32(np.argsort(order).reshape(tokens, k)), torch.from_numpy(w).cuda(), residual=dx)
    torch.cuda.synchronize()
    # each step from the library's own previous one
    mid64, rows64 = to_np(mid), to_np(rows)
    want = x.copy()
    for t in range(tokens):
        for q in range(k):
            want[t] += w[t, q] * rows64[np.argsort(order)[t * k + q]]
    assert (np.abs(to_np(y) - want) <= np.abs(want) * 2.0 ** -8 + 1e-5).all()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        for X, src, got, act in ((A, x[order[lo:hi] // k], mid64, "gelu_tanh"), (B, mid64[lo:hi], rows64, "none")):
            q, s, z, _ = X.quantized(e, src)
            v, dv = R.product_int4(q, s, X.cw[e], X.sw[e], z, X.l2[e], X.bias[e])
            ref, tol = R.epilogue(v, dv, act, out="bf16")
            # z may round to the other bf16 neighbour: one step of it through l2
            tol = tol + 1.13 * (np.abs(R.bf16(z)) * 2.0 ** -7) @ np.abs(X.l2[e]).T
            assert (np.abs(got[lo:hi] - ref) <= tol).all(), e


@pytest.mark.parametrize("seed", range(16))
def test_random_grouped_linears(S, seed):
    rng = np.random.default_rng([11, seed])
    E, n = int(np.exp(rng.uniform(0, np.log(80)))), int(np.exp(rng.uniform(np.log(8), np.log(700))))
    tokens, k = int(np.exp(rng.uniform(0, np.log(300)))), int(rng.integers(1, min(E, 4) + 1))
    m, rank = 64 * int(rng.integers(1, 20)), int(rng.choice([0, 4, 16, 40, 65]))
    act, pad = ["none", "gelu_erf", "silu", "relu"][rng.integers(4)], int(rng.integers(0, 3)) * 7
    _say(f"random grouped E={E} tokens={tokens} k={k} m={m} n={n} rank={rank} {act} pad={pad}")
    X = Experts(S, E, m, n, rank, bias=bool(rng.integers(2)), smooth=bool(rng.integers(2)), seed=seed)
    x = R.bf16(rng.standard_normal((tokens, m)))
    chosen = np.stack([rng.choice(E, k, replace=False) for _ in range(tokens)]).reshape(-1)
    order = np.argsort(chosen, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(chosen, minlength=E))])
    src = np.concatenate([order // k, rng.integers(-3, tokens + 3, pad)])
    b = len(src)
    dx, do, ds = dev_bf16(x), i32(off), i32(src)
    begin = int(rng.integers(0, n + 1))
    y = torch.full((b, n), 99.0, device="cuda")
    S.svdq_grouped_linear(dx, do, X.layer, ds, act=act, act_begin=begin, y=y)
    _, _, z = S.svdq_grouped_quantize_act_lowrank_down(dx, do, X.layer, ds)
    torch.cuda.synchronize()
    got, zz = to_np(y), to_np(z) if rank else np.zeros((b, 0))
    assert (got[off[-1]:] == 99).all()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        codes, s, zr, dz = X.quantized(e, x[src[lo:hi]])
        assert (np.abs(zz[lo:hi] - zr) <= dz + 1e-38).all()
        v, dv = R.product_int4(codes, s, X.cw[e], X.sw[e], zz[lo:hi], X.l2[e], X.bias[e] if X.bias is not None else None)
        want, tol = R.epilogue(v, dv, act, begin)
        assert (np.abs(got[lo:hi] - want) <= tol).all(), e


def test_operands_past_32_bit_offsets(S):
    """Activations and weights of more than 4 GB: rows gathered from the end of x, the last expert's layer."""
    E, m, n, rank = 66, 4096, 32768, 16
    rng = np.random.default_rng(4)
    qw = torch.zeros((E, m // 64, n, 32), dtype=torch.uint8, device="cuda")
    assert qw.numel() > 2 ** 32
    one = Experts(S, 1, m, n, rank, bias=False, smooth=False)
    qw[-1] = one.layer.qw[0]
    wide = lambda t: torch.cat([torch.zeros((E - 1,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda"), t])
    layer = S.GroupedDeviceLayer.from_tensors(E, m, n, rank, qw, wide(one.layer.wscale), wide(one.layer.l1), wide(one.layer.l2))
    rows = 530000
    x = torch.zeros((rows, m), dtype=torch.bfloat16, device="cuda")
    assert x.numel() * 2 > 2 ** 32
    tail = R.bf16(rng.standard_normal((3, m)))
    x[-3:] = dev_bf16(tail)
    src, off = i32([rows - 3, rows - 1, rows - 2]), i32([0] * E + [3])
    y = S.svdq_grouped_linear(x, off, layer, src, out_dtype=torch.float32)
    _, _, z = S.svdq_grouped_quantize_act_lowrank_down(x, off, layer, src)
    torch.cuda.synchronize()
    codes, s, _, _ = one.quantized(0, tail[[0, 2, 1]])
    v, dv = R.product_int4(codes, s, one.cw[0], one.sw[0], to_np(z), one.l2[0])
    want, tol = R.epilogue(v, dv)
    assert (np.abs(to_np(y) - want) <= tol).all()
    # the same rows through the tiles: enough of them that the row kernel is not chosen
    many = i32(np.repeat([rows - 3, rows - 1, rows - 2], 200))
    y = S.svdq_grouped_linear(x, i32([0] * E + [600]), layer, many, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert (np.abs(to_np(y) - np.repeat(want, 200, 0)) <= np.repeat(tol, 200, 0)).all()
