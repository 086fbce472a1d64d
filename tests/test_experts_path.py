"""The experts' path as README writes it, with GELU: forwards with what the way back
needs, and back to the tokens and the router's weights."""
import math

import numpy as np
import pytest

from tests import epi_ref as R
from tests import fp8_ref as F


def gelu(v):
    """(GELU by tanh, its derivative)."""
    c = math.sqrt(2 / math.pi)
    t = np.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)


def forward(x, w1, w2, ids, gate):
    """y and what the way back needs, in 64 bits: tokens' rows by slot (a dropped slot's is not used)."""
    t, k = ids.shape
    y, saved = x.copy(), {}
    for i in range(t):
        for q in range(k):
            e = ids[i, q]
            if e < 0:
                continue
            pre = x[i] @ w1[e]
            mid, slope = gelu(pre)
            row = mid @ w2[e]
            y[i] += gate[i, q] * row
            saved[i, q] = (slope, row)
    return y, saved


def backward(dy, w1, w2, ids, gate, saved):
    dx, dgate = dy.copy(), np.zeros(ids.shape)  # dy: the residual's part
    for (i, q), (slope, row) in saved.items():
        e = ids[i, q]
        dgate[i, q] = dy[i] @ row
        dpre = (gate[i, q] * dy[i]) @ w2[e].T * slope
        dx[i] += dpre @ w1[e].T
    return dx, dgate


def problem(rng, t, k, E, m, h):
    ids = np.array([rng.choice(E, k, replace=False) for _ in range(t)])
    ids[rng.random((t, k)) < 0.1] = -1
    return ids, rng.random((t, k))


def test_formula_against_differences():
    """The steps put together are the gradient (64 bits, central differences)."""
    rng = np.random.default_rng(1)
    t, k, E, m, h = 5, 2, 3, 7, 6
    ids, gate = problem(rng, t, k, E, m, h)
    w1, w2 = rng.standard_normal((E, m, h)), rng.standard_normal((E, h, m))
    x, dy = rng.standard_normal((t, m)), rng.standard_normal((t, m))
    dx, dgate = backward(dy, w1, w2, ids, gate, forward(x, w1, w2, ids, gate)[1])
    step = 1e-5  # central differences: some step^2 of third derivatives, and 2^-52 / step of y
    for i in range(t):
        for j in range(m):
            up, dn = x.copy(), x.copy()
            up[i, j] += step
            dn[i, j] -= step
            d = ((forward(up, w1, w2, ids, gate)[0] - forward(dn, w1, w2, ids, gate)[0]) * dy).sum() / (2 * step)
            assert abs(d - dx[i, j]) < 1e-6
        for q in range(k):
            up, dn = gate.copy(), gate.copy()
            up[i, q] += step
            dn[i, q] -= step
            d = ((forward(x, w1, w2, ids, up)[0] - forward(x, w1, w2, ids, dn)[0]) * dy).sum() / (2 * step)
            assert abs(d - dgate[i, q]) < 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("t,k,E,m,h", [(1, 2, 4, 256, 384), (60, 3, 5, 200, 300)])
def test_readme_path(t, k, E, m, h):
    """Each step of the library on what the step before it left, against the formulas above in 64 bits."""
    torch = pytest.importorskip("torch")
    import w4a4_rank_corrected_amd as S
    rng = np.random.default_rng([t, E])
    ids, gate = problem(rng, t, k, E, m, h)
    gate = gate.astype(np.float32)
    dev = lambda v: torch.from_numpy(R.bf16(v)).to(torch.bfloat16).cuda()
    host = lambda v: v.float().cpu().numpy().astype(np.float64)
    w1, w2 = dev(rng.standard_normal((E, m, h)) / math.sqrt(m)), dev(rng.standard_normal((E, h, m)) / math.sqrt(h))
    x, dy = dev(rng.standard_normal((t, m))), dev(rng.standard_normal((t, m)))
    weight = torch.from_numpy(gate).cuda()

    offsets, row_index, index = S.svdq_sort_rows(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    up, down = S.GroupedDeviceLayerFp8(w1), S.GroupedDeviceLayerFp8(w2)
    pre = S.svdq_fp8_grouped_linear(x, offsets, up, row_index)
    mid = torch.nn.functional.gelu(pre, approximate="tanh")
    rows = S.svdq_fp8_grouped_linear(mid, offsets, down)
    y = S.svdq_combine_rows(rows, index, weight, residual=x)
    drows, dweight = S.svdq_combine_rows_grad(dy, index, weight, rows)
    dmid = S.svdq_fp8_grouped_linear(drows, offsets, S.GroupedDeviceLayerFp8(w2, transposed=True))
    dpre = torch.ops.aten.gelu_backward(dmid, pre, approximate="tanh")
    dtoken = S.svdq_fp8_grouped_linear(dpre, offsets, S.GroupedDeviceLayerFp8(w1, transposed=True))
    dx = S.svdq_combine_rows(dtoken, index, residual=dy)

    off, place = offsets.cpu().numpy(), index.cpu().numpy()
    q1, q2 = ([F.quantize(host(v).T, 128) for v in w] for w in (w1, w2))  # codes of W^T [n][m]

    def product(a, q, back=False):
        q = q[2].T if back else q[2]
        return R.epilogue(*R.product_values(F.quantize(a, 1)[2], q, a.shape[1]), out="bf16")

    half = 2.0 ** -8 * 1.01
    for e in range(E):
        s = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        for got, a, q, back in ((pre, host(x)[row_index.cpu().numpy()[s]], q1[e], False), (rows, host(mid)[s], q2[e], False),
                                (dmid, host(drows)[s], q2[e], True), (dtoken, host(dpre)[s], q1[e], True)):
            v, bound = product(a, q, back)
            assert (np.abs(host(got)[s] - v) <= bound).all()
        g, slope = gelu(host(pre)[s])
        # torch's own evaluation in 32 bits: some units of rounding of terms of at most |v| and |dmid|, then bf16's
        assert (np.abs(host(mid)[s] - g) <= np.abs(g) * half + 64 * R.U * np.abs(host(pre)[s])).all()
        want = host(dmid)[s] * slope
        assert (np.abs(host(dpre)[s] - want) <= np.abs(want) * half + 256 * R.U * np.abs(host(dmid)[s])).all()
    want, size = host(x).copy(), np.abs(host(x))
    back, bsize = host(dy).copy(), np.abs(host(dy))  # the residual's gradient is dy
    for i in range(t):
        for q in range(k):
            r = place[i, q]
            if r < 0:
                assert float(dweight[i, q]) == 0
                continue
            term = gate[i, q].astype(np.float64) * host(rows[r])
            want[i] += term
            size[i] += np.abs(term)
            back[i] += host(dtoken[r])
            bsize[i] += np.abs(host(dtoken[r]))
            prod = host(dy[i]) * host(rows[r])
            assert abs(float(dweight[i, q]) - prod.sum()) <= (m + 8) * R.U * np.abs(prod).sum()
            d = gate[i, q].astype(np.float64) * host(dy[i])
            assert (np.abs(host(drows[r]) - d) <= np.abs(d) * (half + R.U)).all()
    assert (np.abs(host(y) - want) <= (k + 2) * 2 * R.U * size + np.abs(want) * half).all()
    assert (np.abs(host(dx) - back) <= (k + 2) * 2 * R.U * bsize + np.abs(back) * half).all()
