"""The gradient of the combination of rows over every index that the combination
takes: rows that no slot names, slots that name no row, rows that several name."""
import numpy as np
import pytest

from tests import epi_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a4_rank_corrected_amd as S
    S.lib()
    return S


def dt(out):
    return torch.bfloat16 if out == "bf16" else torch.float32


def data(rng, shape, out):
    v = rng.standard_normal(shape)
    v = R.bf16(v) if out == "bf16" else v.astype(np.float32).astype(np.float64)
    return v, torch.from_numpy(v).to(dt(out)).cuda()


def reference(dy, rows, index, w):
    """(drows, the sums of their terms' magnitudes, terms of each row, dweight, the sums of its terms' magnitudes)."""
    Rn, n = rows.shape
    d, size, terms = np.zeros((Rn, n)), np.zeros((Rn, n)), np.zeros(Rn, int)
    t, q = np.nonzero((index >= 0) & (index < Rn))
    r = index[t, q]
    c = np.ones(len(t)) if w is None else w[t, q].astype(np.float64)
    np.add.at(d, r, c[:, None] * dy[t])
    np.add.at(size, r, np.abs(c[:, None] * dy[t]))
    np.add.at(terms, r, 1)
    dw, ds = np.zeros(index.shape), np.zeros(index.shape)
    dw[t, q] = (dy[t] * rows[r]).sum(1)
    ds[t, q] = np.abs(dy[t] * rows[r]).sum(1)
    return d, size, terms, dw, ds


def check(S, index, Rn, n, out, weighted, seed, unaligned=False):
    rng = np.random.default_rng(seed)
    t, k = index.shape
    dy, dyd = data(rng, (t, n), out)
    rows, rd = data(rng, (Rn, n), out)
    w = rng.standard_normal((t, k)).astype(np.float32) if weighted else None
    wd = torch.from_numpy(w).cuda() if weighted else None
    idx = torch.zeros(t * k + 1, dtype=torch.int32).cuda()[1 if unaligned else 0:][: t * k].view(t, k)
    idx.copy_(torch.from_numpy(index.astype(np.int32)))
    d, size, terms, dw, ds = reference(dy, rows, index, w)
    guard = torch.full((Rn + 2, n), float("nan"), dtype=dt(out)).cuda()
    drows, dweight = S.svdq_combine_rows_grad(dyd, idx, wd, rd, drows=guard[1: 1 + Rn])
    got = drows.float().cpu().numpy().astype(np.float64)
    # each product is off by half a step, u, each of terms - 1 additions by u of the magnitudes added so far, and the
    # result's rounding by half a step of y's
    half = 2.0 ** -8 if out == "bf16" else 0.0
    bound = np.maximum(terms, 1)[:, None] * R.U * 1.01 * size + np.abs(d) * half * 1.01 + 1e-38
    assert (np.abs(got - d) <= bound).all()
    assert (got[terms == 0] == 0).all()
    assert torch.isnan(guard[0]).all() and torch.isnan(guard[-1]).all()
    if not weighted:
        one = terms == 1
        assert np.array_equal(got[one], d[one])
    assert (np.abs(dweight.cpu().numpy() - dw) <= (n + 8) * R.U * ds).all()
    assert (dweight.cpu().numpy()[(index < 0) | (index >= Rn)] == 0).all()
    # the same again, each output alone, and in place on the rows
    for _ in range(2):
        d2, w2 = S.svdq_combine_rows_grad(dyd, idx, wd, rd)
        assert torch.equal(d2, drows) and torch.equal(w2, dweight)
    only, none = S.svdq_combine_rows_grad(dyd, idx, wd, drows=torch.full_like(rd, float("nan")))
    assert none is None and torch.equal(only, drows)
    own = rd.clone()
    d3, w3 = S.svdq_combine_rows_grad(dyd, idx, wd, own, drows=own)
    assert d3.data_ptr() == own.data_ptr() and torch.equal(d3, drows) and torch.equal(w3, dweight)


def test_rows_that_no_slot_names_have_no_gradient(S):
    """A row buffer with unused rows at its end and between (no row is named twice, and none by a negative index)."""
    index = np.array([[3, 7], [1, 30], [12, 5], [40, 9]])  # 30 and 40: outside the 16 rows
    check(S, index, 16, 70, "bf16", True, 0)
    check(S, index, 16, 70, "f32", False, 0)


@pytest.mark.parametrize("t,k,Rn,n", [(1, 1, 1, 1), (1, 1, 3, 5), (3, 2, 9, 77), (5, 3, 4, 130), (40, 4, 200, 264), (33, 7, 50, 1153),
                                      (300, 6, 1500, 100), (700, 2, 5003, 40), (64, 1, 20, 2500), (9, 2, 18, 9000)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
def test_any_index(S, t, k, Rn, n, out, weighted):
    """Rows named by none, one and several slots; -1 and other values outside the rows, which name none."""
    print(f"grad t={t} k={k} R={Rn} n={n} {out} weighted={weighted}", flush=True)
    rng = np.random.default_rng([t, k, Rn, n])
    index = rng.integers(-2, Rn + 2, (t, k))
    index.reshape(-1)[::5] = rng.choice([-1, -1 - Rn, Rn, 2 ** 31 - 1, -2 ** 31], len(index.reshape(-1)[::5]))
    index.reshape(-1)[0] = 0  # beside the -1s, which stand for no row
    check(S, index, Rn, n, out, weighted, [t, k, Rn, n], unaligned=n % 2 == 1)


@pytest.mark.parametrize("kind", ["all one", "two rows", "long lists", "more than a workgroup lists", "mean 6"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_rows_of_many_slots(S, kind, out):
    rng = np.random.default_rng(7)
    t, k, Rn, n = 1300, 5, 40, 70
    if kind == "all one":
        index = np.full((t, k), 11)
    elif kind == "two rows":
        index = rng.choice([0, 39], (t, k))
    elif kind == "long lists":  # about the lengths at which a list is given up
        c = np.repeat(np.arange(40), 30 + 2 * np.arange(40))[: t * k]
        index = np.concatenate([rng.permutation(c), np.full(t * k - len(c), -1)]).reshape(t, k)
    elif kind == "mean 6":
        Rn = t * k // 6
        index = rng.integers(0, Rn, (t, k))
    else:  # ten rows a workgroup (of 512), 60 slots each, in some of them more
        Rn, t, k, n = 5120, 60000, 5, 8
        index = rng.integers(0, Rn, (t, k))
        index[:20000] = rng.integers(0, 40, (20000, k))
    check(S, index, Rn, n, out, True, 3)


def test_no_tokens_and_no_rows(S):
    w = torch.empty(0, 2).cuda()
    rows = torch.full((5, 8), 3.0).cuda()
    drows, dweight = S.svdq_combine_rows_grad(torch.empty(0, 8).cuda(), torch.empty(0, 2, dtype=torch.int32).cuda(), w, rows)
    assert drows.shape == (5, 8) and (drows == 0).all() and dweight.shape == (0, 2)
    drows, dweight = S.svdq_combine_rows_grad(torch.ones(3, 8).cuda(), torch.zeros(3, 2, dtype=torch.int32).cuda(), None,
                                              torch.empty(0, 8).cuda())
    assert drows.shape == (0, 8) and (dweight == 0).all()


def test_against_differences(S):
    """combine is linear in the rows and in the weights: its change along one entry is the gradient's, up to the sums'
    own rounding, which the entries of one token's sums bound."""
    rng = np.random.default_rng(4)
    t, k, Rn, n = 30, 3, 70, 200
    index = rng.integers(-1, 50, (t, k))  # rows 50 .. 69 are not named
    index[7] = [4, 4, -1]
    idx = torch.from_numpy(index.astype(np.int32)).cuda()
    rows, dy = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda() for s in ((Rn, n), (t, n)))
    w = torch.from_numpy((0.25 + rng.random((t, k))).astype(np.float32)).cuda()
    y = lambda r, v: S.svdq_combine_rows(r, idx, v).double()
    drows, dweight = S.svdq_combine_rows_grad(dy, idx, w, rows)
    h = 0.5
    u = R.U

    def compare(up, dn, g, step, scale):
        """step: the entry's change; scale: |dy| summed against the magnitudes of the entries of y that change."""
        diff = float(((up - dn) * dy.double()).sum()) / step
        # two sums of at most k products each, off by (k + 1) u of their magnitudes; the gradient itself by n + 8 of them
        tol = 2 * (k + 2) * u * scale / step + 2 * (n + 8) * u * scale
        assert abs(diff - g) <= tol, (diff, g, tol)
        return tol

    big = 0
    for r, j in [(4, 5), (index[0, 0] % 50, 0), (49, n - 1), (60, 3)]:
        up, dn = rows.clone(), rows.clone()
        up[r, j] += h
        dn[r, j] -= h
        step = float(up[r, j].double() - dn[r, j].double())
        named = np.nonzero((index == r).any(1))[0]
        scale = sum(float(dy[i, j].abs()) * float((w[i] * (rows[idx[i].clamp(min=0).long(), j].abs() + h)).sum()) for i in named)
        g = float(drows[r, j])
        if compare(y(up, w), y(dn, w), g, step, scale) * 100 < abs(g):
            big += 1
    for i, q in [(7, 0), (7, 1), (0, 0), (3, 2)]:
        up, dn = w.clone(), w.clone()
        up[i, q] += h
        dn[i, q] -= h
        step = float(up[i, q].double() - dn[i, q].double())
        scale = float((dy[i].abs() * ((w[i, :, None] + h) * rows[idx[i].clamp(min=0).long()].abs()).sum(0)).sum())
        g = float(dweight[i, q])
        if compare(y(rows, up), y(rows, dn), g, step, scale) * 100 < abs(g):
            big += 1
    assert big >= 4  # gradients a hundred times the tolerance


def test_captured_and_replayed(S):
    t, k, Rn, n = 90, 4, 300, 264
    rng = np.random.default_rng(1)
    sets = []
    for i in range(4):
        index = torch.from_numpy(rng.integers(-1, Rn, (t, k)).astype(np.int32)).cuda()
        sets.append((torch.randn(t, n).bfloat16().cuda(), index, torch.rand(t, k).cuda(), torch.randn(Rn, n).bfloat16().cuda()))
    want = [[v.clone() for v in S.svdq_combine_rows_grad(*s)] for s in sets]
    inputs = [v.clone() for v in sets[0]]
    dr, dw = torch.empty(Rn, n, dtype=torch.bfloat16).cuda(), torch.empty(t, k).cuda()
    S.svdq_combine_rows_grad(*inputs, drows=dr, dweight=dw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.svdq_combine_rows_grad(*inputs, drows=dr, dweight=dw)
    for i in (1, 2, 3, 0, 2):
        for a, b in zip(inputs, sets[i]):
            a.copy_(b)
        dr.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dr, want[i][0]) and torch.equal(dw, want[i][1]), i
        assert torch.equal(S.svdq_combine_rows_grad(*sets[i])[0], want[i][0])


@pytest.mark.parametrize("Rn", [270001, (1 << 22)])
def test_most_rows(S, Rn):
    """Workgroups of many rows, and of the most there are."""
    rng = np.random.default_rng(Rn)
    index = rng.integers(-1, Rn, (200000, 4))
    index[1000] = index[1001]
    check(S, index, Rn, 2, "f32", True, 5)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_rows_past_32_bit_offsets(S, out):
    """Rows of more than 4 GB: the gradients and the dispatch of the first and the last ones."""
    n, t, k = 4096, 40, 3
    Rn = 300000 if out == "f32" else 600000
    rng = np.random.default_rng(3)
    at = np.concatenate([rng.choice(50, 60, replace=True), Rn - 1 - rng.choice(50, 60, replace=True)])
    index = rng.permutation(at).reshape(t, k)
    rows = torch.zeros(Rn, n, dtype=dt(out), device="cuda")
    used = np.unique(index)
    some, sd = data(rng, (len(used), n), out)
    rows[torch.from_numpy(used).cuda()] = sd
    dy, dyd = data(rng, (t, n), out)
    idx = torch.from_numpy(index.astype(np.int32)).cuda()
    place = np.searchsorted(used, index)
    d, size, terms, dw, ds = reference(dy, some, place, None)
    drows, dweight = S.svdq_combine_rows_grad(dyd, idx, None, rows, drows=torch.full_like(rows, float("nan")))
    got = drows[torch.from_numpy(used).cuda()].float().cpu().numpy().astype(np.float64)
    half = 2.0 ** -8 if out == "bf16" else 0.0
    assert (np.abs(got - d) <= terms[:, None] * R.U * 1.01 * size + np.abs(d) * half * 1.01).all()
    assert (np.abs(dweight.cpu().numpy() - dw) <= (n + 8) * R.U * ds).all()
    drows[torch.from_numpy(used).cuda()] = 0
    for lo in range(0, Rn, 50000):
        assert (drows[lo: lo + 50000] == 0).all()  # all the others were made zero
    once, first = np.unique(index, return_index=True)
    single = np.full((t, k), Rn, np.int64)  # each row once: what dispatch takes
    single.reshape(-1)[first] = once
    drows.fill_(7)
    S.svdq_dispatch_rows(dyd, torch.from_numpy(single.astype(np.int32)).cuda(), rows=drows)
    assert torch.equal(drows[torch.from_numpy(once).cuda()], dyd[torch.from_numpy(first // k).cuda()])
    assert (drows[Rn // 2 - 100: Rn // 2 + 100] == 7).all()
