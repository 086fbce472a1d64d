"""The routing of rows to experts on the GPU: the sort exactly, the dispatch and
the combination's gradient against 64-bit references, and whole runs of the
experts' path forwards and backwards."""
import sys

import numpy as np
import pytest

from tests import epi_ref as R
from tests import fp8_ref as F

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


def to_dev(v, out):
    return dev_bf16(v) if out == "bf16" else torch.from_numpy(np.asarray(v, np.float32)).cuda()


def values(v, out):
    return R.bf16(v) if out == "bf16" else np.asarray(v, np.float32).astype(np.float64)


def sorted_slots(ids, E):
    t, k = ids.shape
    key = np.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    order = np.argsort(key, kind="stable")
    place = np.empty(t * k, int)
    place[order] = np.arange(t * k)
    index = np.where(key < E, place, -1 - place).reshape(t, k)
    return np.searchsorted(key[order], np.arange(E + 1)), order // k, index


def choose(rng, t, k, E, dropped=0.1):
    ids = rng.integers(0, E, (t, k))
    ids[rng.random((t, k)) < dropped] = -1
    return ids


# ---------------------------------------------------------------------------
# sort
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("t,k,E", [(1, 1, 1), (1, 2, 16), (5, 3, 2), (32, 4, 64), (100, 6, 63), (511, 1, 65), (700, 6, 128),
                                   (683, 6, 8), (4097, 1, 3), (3001, 6, 64), (9000, 8, 255), (4096, 2, 1024), (65536, 3, 1000)])
@pytest.mark.parametrize("kind", ["some", "all one", "all dropped", "any"])
def test_sort(S, t, k, E, kind):
    _say(f"sort t={t} k={k} E={E} {kind}")
    rng = np.random.default_rng([t, k, E])
    ids = choose(rng, t, k, E)
    if kind == "all one":
        ids[:] = E - 1
    elif kind == "all dropped":
        ids[:] = E
    elif kind == "any":  # any 32-bit value
        ids = rng.integers(-2 ** 31, 2 ** 31, (t, k))
        ids[0] = E // 2
    off, row, index = S.svdq_sort_rows(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    o, r, x = sorted_slots(ids.astype(np.int32).astype(np.int64), E)
    assert np.array_equal(off.cpu().numpy(), o)
    assert np.array_equal(row.cpu().numpy(), r)
    assert np.array_equal(index.cpu().numpy(), x)


def test_sort_largest(S):
    """The most slots there can be: chunks of more than 8 slots a thread."""
    t, k, E = (1 << 22) // 4, 4, 300
    ids = torch.randint(-1, E, (t, k), dtype=torch.int32, device="cuda")
    off, row, index = S.svdq_sort_rows(ids, E)
    o, r, x = sorted_slots(ids.cpu().numpy().astype(np.int64), E)
    assert np.array_equal(off.cpu().numpy(), o) and np.array_equal(row.cpu().numpy(), r)
    assert np.array_equal(index.cpu().numpy(), x)


def test_sort_no_tokens(S):
    off, row, index = S.svdq_sort_rows(torch.empty(0, 3, dtype=torch.int32).cuda(), 70)
    assert (off == 0).all() and off.numel() == 71 and row.numel() == 0 and index.shape == (0, 3)


# ---------------------------------------------------------------------------
# dispatch and the combination's gradient
# ---------------------------------------------------------------------------

CASES = [(1, 1, 1), (3, 2, 8), (7, 2, 77), (7, 3, 1153), (40, 9, 264), (5, 20, 1152), (64, 1, 2048), (300, 6, 100), (2500, 2, 40),
         (3, 4, 5000)]


@pytest.mark.parametrize("t,k,n", CASES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_and_grad(S, t, k, n, out, weighted):
    _say(f"dispatch and grad t={t} k={k} n={n} {out} weighted={weighted}")
    rng = np.random.default_rng([t, k, n])
    index = sorted_slots(choose(rng, t, k, 16), 16)[2]
    x, rows = values(rng.standard_normal((t, n)), out), values(rng.standard_normal((t * k, n)), out)
    w = rng.standard_normal((t, k)).astype(np.float32)
    w.reshape(-1)[0] = 0
    idx, wd = torch.from_numpy(index.astype(np.int32)).cuda(), torch.from_numpy(w).cuda() if weighted else None
    xd, rd = to_dev(x, out), to_dev(rows, out)
    want = np.zeros((t * k, n))
    dw, dsum = np.zeros((t, k)), np.zeros((t, k))
    for i in range(t):
        for q in range(k):
            if index[i, q] >= 0:
                want[index[i, q]] = x[i] * (float(w[i, q]) if weighted else 1.0)
                dw[i, q] = (x[i] * rows[index[i, q]]).sum()
                dsum[i, q] = np.abs(x[i] * rows[index[i, q]]).sum()
    got = S.svdq_dispatch_rows(xd, idx, wd)
    # the fp32 product (half a step), then the output's rounding (half a step of its own)
    half = (2.0 ** -8 if out == "bf16" else 0) + R.U
    assert (np.abs(to_np(got) - want) <= np.abs(want) * half * 1.01 + 1e-38).all()
    if not weighted:
        assert np.array_equal(to_np(got), want)
    drows, dweight = S.svdq_combine_rows_grad(xd, idx, wd, rd)
    assert torch.equal(drows, got)
    # n products and as many additions of a tree, each half a step of at most the sum of the magnitudes
    assert (np.abs(to_np(dweight) - dw) <= (n + 8) * R.U * dsum).all()
    assert (dweight.cpu().numpy()[index < 0] == 0).all()
    # each output by itself, and in place on the rows
    only, none = S.svdq_combine_rows_grad(xd, idx, wd)
    assert none is None and torch.equal(only, got)
    own = rd.clone()
    d2, w2 = S.svdq_combine_rows_grad(xd, idx, wd, own, drows=own)
    assert d2.data_ptr() == own.data_ptr() and torch.equal(d2, got) and torch.equal(w2, dweight)


def test_grad_is_the_transpose_of_the_combination(S):
    """<dy, combine(rows)> = <drows, rows> = sum w dw, and differences along one row and one weight."""
    rng = np.random.default_rng(4)
    t, k, n = 30, 3, 200
    index = sorted_slots(choose(rng, t, k, 5), 5)[2]
    idx = torch.from_numpy(index.astype(np.int32)).cuda()
    rows, dy = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda() for s in ((t * k, n), (t, n)))
    w = torch.from_numpy(rng.random((t, k)).astype(np.float32)).cuda()
    loss = lambda r, v: float((S.svdq_combine_rows(r, idx, v).double() * dy.double()).sum())
    drows, dweight = S.svdq_combine_rows_grad(dy, idx, w, rows)
    # rows are below 5 and weights below 1: a sum of k of them is below 16 and off by (k + 1) u of that at most
    total = float(dy.double().abs().sum() * 4)
    tol = (k + 8) * 2 * R.U * total * 4
    assert abs(loss(rows, w) - float((drows.double() * rows.double()).sum())) <= tol
    assert abs(loss(rows, w) - float((dweight.double() * w.double()).sum())) <= tol + (n + 8) * R.U * total * 4
    h = 0.5  # linear in each: any step serves
    for q in (0, 1, 2):
        up, dn = w.clone(), w.clone()
        up[7, q] += h
        dn[7, q] -= h
        assert abs((loss(rows, up) - loss(rows, dn)) / (2 * h) - float(dweight[7, q])) <= tol / h
    for r, j in ((0, 0), (11, 5), (t * k - 1, n - 1)):
        up, dn = rows.clone(), rows.clone()
        up[r, j] += h
        dn[r, j] -= h
        assert abs((loss(up, w) - loss(dn, w)) / (2 * h) - float(drows[r, j])) <= tol / h


def test_rows_that_are_not_there(S):
    """Indexes outside the rows write nothing and have no gradient; rows that no slot names stay as they were."""
    t, k, n, R_ = 4, 3, 130, 9
    index = np.array([[0, -1 - 4, 9], [2, -1 - 9, 1 << 30], [-(1 << 31), 7, -1 - 8], [3, 5, 2 ** 31 - 1]])
    idx = torch.from_numpy(index.astype(np.int32)).cuda()
    x = torch.randn(t, n).cuda()
    guard = torch.full((R_ + 4, n), 6.0).cuda()
    S.svdq_dispatch_rows(x, idx, rows=guard[2: 2 + R_])
    want = torch.full((R_, n), 6.0).cuda()
    for r, i in ((0, 0), (2, 1), (7, 2), (3, 3), (5, 3)):
        want[r] = x[i]
    want[4] = want[8] = 0
    assert torch.equal(guard[2: 2 + R_], want) and (guard[:2] == 6).all() and (guard[2 + R_:] == 6).all()
    rows = torch.full((R_, n), float("nan")).cuda()  # rows that are not named are not read
    for r in (0, 2, 7, 3, 5):
        rows[r] = 1.0
    _, dw = S.svdq_combine_rows_grad(x, idx, None, rows)
    named = torch.from_numpy((index >= 0) & (index < R_)).cuda()
    assert (dw[~named] == 0).all()
    assert torch.allclose(dw[named], x.sum(1, keepdim=True).expand(-1, k)[named], rtol=0, atol=float(n * R.U * 8 * n))


def test_unaligned_and_nonfinite(S):
    for out in ("f32", "bf16"):
        dt = torch.float32 if out == "f32" else torch.bfloat16
        t, k, n = 9, 2, 333
        rng = np.random.default_rng(1)
        index = sorted_slots(choose(rng, t, k, 4), 4)[2]
        idx = torch.from_numpy(index.astype(np.int32)).cuda()
        base = [torch.randn(t * n + 1).to(dt).cuda(), torch.randn(t * k * n + 3).to(dt).cuda(), torch.zeros(t * k * n + 1, dtype=dt).cuda()]
        x, rows, dr = base[0][1:].view(t, n), base[1][3:].view(t * k, n), base[2][1:].view(t * k, n)
        w = torch.rand(t, k).cuda()
        want = S.svdq_combine_rows_grad(x.clone(), idx, w, rows.clone())
        got = S.svdq_combine_rows_grad(x, idx, w, rows, drows=dr)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # a NaN token reaches its own rows and weights only; a dropped slot's row stays zero
        xn = x.clone()
        xn[4] = float("nan")
        dn, wn = S.svdq_combine_rows_grad(xn, idx, w, rows)
        hit = torch.zeros(t * k, dtype=torch.bool).cuda()
        hit[idx[4][idx[4] >= 0].long()] = True
        assert torch.isnan(dn[hit]).all() and torch.equal(dn[~hit], want[0][~hit])
        assert torch.equal(wn[torch.arange(t) != 4], want[1][torch.arange(t) != 4])
        assert (wn[4][idx[4] < 0] == 0).all()


# ---------------------------------------------------------------------------
# whole runs
# ---------------------------------------------------------------------------

class Net:
    """Two layers an expert, tokens through their experts and back: forward, and the gradients of tokens and weights."""

    def __init__(self, S, E, m, hidden, seed):
        rng = np.random.default_rng(seed)
        self.E, self.m, self.h, self.S = E, m, hidden, S
        w1, w2 = R.bf16(rng.standard_normal((E, hidden, m)) / np.sqrt(m)), R.bf16(rng.standard_normal((E, m, hidden)) / np.sqrt(hidden))
        self.q1, self.q2 = ([F.quantize(v, 128) for v in w] for w in (w1, w2))
        d1, d2 = dev_bf16(w1), dev_bf16(w2)
        self.fc1, self.fc2 = (S.GroupedDeviceLayerFp8(d, transposed=True) for d in (d1, d2))
        self.bc1, self.bc2 = (S.GroupedDeviceLayerFp8(d) for d in (d1, d2))  # of the transposes

    @staticmethod
    def layer(x, q, transpose=False, tiles=False):
        """(v, bound) of rows x through a layer's quantize() result (or its transpose's)."""
        xq = F.quantize(x, 1)
        if transpose:
            q = tuple(a.T for a in q)
        v, dv = R.product_values(xq[2], q[2], x.shape[1])
        return v, dv + F.aligned(xq, q) if tiles else dv

    def forward(self, x, ids, gate):
        S = self.S
        off, row, index = S.svdq_sort_rows(ids, self.E)
        mid = S.svdq_fp8_grouped_linear(x, off, self.fc1, row, act="relu", y=torch.zeros(row.numel(), self.h, dtype=torch.bfloat16, device="cuda"))
        rows = S.svdq_fp8_grouped_linear(mid, off, self.fc2, y=torch.zeros(row.numel(), self.m, dtype=torch.bfloat16, device="cuda"))
        y = S.svdq_combine_rows(rows, index, gate, residual=x)
        return y, (off, row, index, mid, rows)

    def backward(self, dy, gate, saved):
        S = self.S
        off, row, index, mid, rows = saved
        drows, dgate = S.svdq_combine_rows_grad(dy, index, gate, rows)
        dmid = S.svdq_fp8_grouped_linear(drows, off, self.bc2, y=torch.zeros_like(mid))
        dmid = torch.where(mid > 0, dmid, torch.zeros_like(dmid))
        din = S.svdq_fp8_grouped_linear(dmid, off, self.bc1, y=torch.zeros(row.numel(), self.m, dtype=torch.bfloat16, device="cuda"))
        dx = S.svdq_combine_rows(din, index, residual=dy)
        return dx, dgate


@pytest.mark.parametrize("t,k,E,m,hidden", [(1, 2, 4, 256, 384), (50, 2, 6, 200, 300), (333, 3, 8, 256, 130)])
def test_experts_forwards_and_backwards(S, t, k, E, m, hidden):
    """Every step of the run, each on what the step before it left, against the formulas in 64 bits."""
    _say(f"experts' path t={t} k={k} E={E} m={m} hidden={hidden}")
    rng = np.random.default_rng([t, k, E])
    net = Net(S, E, m, hidden, [t, E])
    ids = choose(rng, t, k, E)
    x, gate = R.bf16(rng.standard_normal((t, m))), rng.random((t, k)).astype(np.float32)
    dy = R.bf16(rng.standard_normal((t, m)))
    gd = torch.from_numpy(gate).cuda()
    tiles = t * k > 64 * E
    y, saved = net.forward(dev_bf16(x), torch.from_numpy(ids.astype(np.int32)).cuda(), gd)
    dx, dgate = net.backward(dev_bf16(dy), gd, saved)
    off, row, index = sorted_slots(ids, E)
    assert np.array_equal(saved[0].cpu().numpy(), off) and np.array_equal(saved[2].cpu().numpy(), index)
    mid, rows = to_np(saved[3]), to_np(saved[4])
    for e in range(E):
        s = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        yv, b = R.epilogue(*net.layer(x[row[s]], net.q1[e], tiles=tiles), "relu", out="bf16")
        assert (np.abs(mid[s] - yv) <= b).all()
        yv, b = R.epilogue(*net.layer(mid[s], net.q2[e], tiles=tiles), out="bf16")
        assert (np.abs(rows[s] - yv) <= b).all()
    want = x.copy()
    size = np.abs(x)
    for q in range(k):
        on = index[:, q] >= 0
        want[on] += gate[on, q: q + 1] * rows[index[on, q]]
        size[on] += np.abs(gate[on, q: q + 1] * rows[index[on, q]])
    assert (np.abs(to_np(y) - want) <= (k + 1) * R.U * size + np.abs(want) * 2.0 ** -8 * 1.01).all()
    # backwards
    drows = np.zeros((t * k, m))
    dg, ds = np.zeros((t, k)), np.zeros((t, k))
    for q in range(k):
        on = index[:, q] >= 0
        drows[index[on, q]] = R.bf16((gate[on, q: q + 1] * dy[on].astype(np.float32)).astype(np.float32))
        dg[on, q] = (dy[on] * rows[index[on, q]]).sum(1)
        ds[on, q] = np.abs(dy[on] * rows[index[on, q]]).sum(1)
    assert (np.abs(to_np(dgate) - dg) <= (m + 8) * R.U * ds).all()
    want, size = dy.copy(), np.abs(dy)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        dm, bm = R.epilogue(*net.layer(drows[s], net.q2[e], True, tiles), out="bf16")
        got = S.svdq_fp8_grouped_linear(dev_bf16(drows), saved[0], net.bc2, y=torch.zeros_like(saved[3]))
        assert (np.abs(to_np(got)[s] - dm) <= bm).all()
        g = np.where(mid[s] > 0, to_np(got)[s], 0)
        di, bi = R.epilogue(*net.layer(g, net.q1[e], True, tiles), out="bf16")
        want_rows = di  # (the token's sum below takes the library's own rounding of these: within bi of them)
        for r in range(off[e], off[e + 1]):
            want[row[r]] += want_rows[r - off[e]]
            size[row[r]] += np.abs(want_rows[r - off[e]]) + bi[r - off[e]] / R.U / 4
    # |dx - want| <= the rows' own bounds (in size, times 4 u) + the additions' + one rounding
    assert (np.abs(to_np(dx) - want) <= (k + 4) * R.U * size + np.abs(want) * 2.0 ** -8 * 1.02).all()


def test_int4_experts_take_the_sort(S):
    """The INT4 grouped layer and the combination on the sort's plan, against single tokens."""
    E, m, n, t, k = 5, 128, 96, 21, 2
    rng = np.random.default_rng(0)
    qw = torch.from_numpy(rng.integers(0, 256, (E, m // 64, n, 32)).astype(np.uint8)).cuda()
    ws = torch.full((E, m // 64, n), 0.01, dtype=torch.float16).cuda()
    lay = S.GroupedDeviceLayer.from_tensors(E, m, n, 0, qw, ws)
    x = dev_bf16(R.bf16(rng.standard_normal((t, m))))
    ids = torch.from_numpy(choose(rng, t, k, E).astype(np.int32)).cuda()
    off, row, index = S.svdq_sort_rows(ids, E)
    rows = S.svdq_grouped_linear(x, off, lay, row, out_dtype=torch.float32)
    y = S.svdq_combine_rows(rows, index)
    for i in range(t):
        o1, r1, i1 = S.svdq_sort_rows(ids[i: i + 1].contiguous(), E)
        want = S.svdq_combine_rows(S.svdq_grouped_linear(x[i: i + 1].contiguous(), o1, lay, r1, out_dtype=torch.float32), i1)
        assert torch.allclose(y[i: i + 1], want, rtol=0, atol=1e-4)


def test_graph_of_the_whole_path(S):
    """Forward and backward captured once, replayed with new tokens and routing between eager calls."""
    t, k, E, m, hidden = 40, 2, 6, 256, 200
    net = Net(S, E, m, hidden, 3)
    rng = np.random.default_rng(2)
    sets = [(dev_bf16(R.bf16(rng.standard_normal((t, m)))), torch.from_numpy(choose(rng, t, k, E).astype(np.int32)).cuda(),
             torch.from_numpy(rng.random((t, k)).astype(np.float32)).cuda(), dev_bf16(R.bf16(rng.standard_normal((t, m)))))
            for _ in range(4)]

    def run(x, ids, gate, dy):
        y, saved = net.forward(x, ids, gate)
        dx, dgate = net.backward(dy, gate, saved)
        return y, dx, dgate

    want = [[v.clone() for v in run(*s)] for s in sets]
    torch.cuda.synchronize()
    inputs = [v.clone() for v in sets[0]]
    run(*inputs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run(*inputs)
    for i in (1, 2, 3, 0, 2):
        for a, b in zip(inputs, sets[i]):
            a.copy_(b)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want[i]):
            assert torch.equal(a, b), i
        assert all(torch.equal(a, b) for a, b in zip(run(*sets[i]), want[i]))


@pytest.mark.parametrize("t", [30, 3000])
def test_sorts_on_two_streams(S, t):
    rng = np.random.default_rng(t)
    k, E = 4, 50
    ids = [torch.from_numpy(choose(rng, t, k, E).astype(np.int32)).cuda() for _ in range(2)]
    want = [[v.clone() for v in S.svdq_sort_rows(i, E)] for i in ids]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [S.svdq_sort_rows(i, E, stream=s) for i, s in zip(ids, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
