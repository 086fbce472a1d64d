"""CPU tests of the 8-bit floating-point setting and of the routing of rows: every
refusal of the C ABI and of the binding, the workspaces asked for, and the
reference's own quantizer.  No test here launches a kernel."""
import ctypes
import os

import numpy as np
import pytest

from tests import fp8_ref as F

S = pytest.importorskip("w4a4_rank_corrected_amd")
from w4a4_rank_corrected_amd import _binding as B  # noqa: E402

FAKE = 0x10000      # never dereferenced: every call below is refused (or has nothing to do)
FAR = 0x40000000    # apart from FAKE by more than any tensor here
FAR2 = 0x80000000
INVALID, UNSUPPORTED, ALIGN, WS = (B.SVDQ_ERR_INVALID_ARG, B.SVDQ_ERR_UNSUPPORTED, B.SVDQ_ERR_ALIGNMENT,
                                   B.SVDQ_ERR_WORKSPACE)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libsvdq.so not built")
    return B.lib()


def layer(**kw):
    d = dict(m=200, n=64, qw=FAKE, wscale=FAKE, bias=None)
    d.update(kw)
    d.pop("experts", None)
    return ctypes.byref(B.svdq_fp8_layer(d["m"], d["n"], d["qw"], d["wscale"], d["bias"]))


def grouped(**kw):
    d = dict(experts=4, m=200, n=64, qw=FAKE, wscale=FAKE, bias=None)
    d.update(kw)
    return ctypes.byref(B.svdq_fp8_grouped_layer(d["experts"], d["m"], d["n"], d["qw"], d["wscale"], d["bias"]))


def epi(act=0, act_begin=0, gate_rows=0, ldr=0, ldy=0, gate=None, residual=None):
    return ctypes.byref(B.svdq_epilogue(act, act_begin, gate_rows, ldr, ldy, gate, residual))


BAD_LAYERS = [(dict(m=0), INVALID), (dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(m=B.SVDQ_MAX_DIM + 1), UNSUPPORTED),
              (dict(n=B.SVDQ_MAX_DIM + 1), UNSUPPORTED), (dict(qw=None), INVALID), (dict(qw=FAKE + 8), ALIGN),
              (dict(wscale=None), INVALID), (dict(bias=FAKE + 1), ALIGN)]


@pytest.mark.parametrize("kw,code", BAD_LAYERS)
def test_layer_refusals(L, kw, code):
    assert L.svdq_fp8_gemm(FAKE, FAKE, layer(**kw), None, 16, FAKE, 0, FAKE, BIG, None) == code
    assert L.svdq_last_error()
    assert L.svdq_fp8_linear(FAKE, layer(**kw), None, 16, FAKE, 0, FAKE, BIG, None) == code
    assert L.svdq_fp8_grouped_gemm(FAKE, FAKE, 16, None, FAKE, grouped(**kw), None, 16, FAKE, 0, None) == code
    assert L.svdq_fp8_grouped_linear(FAKE, 16, None, FAKE, grouped(**kw), None, 16, FAKE, 0, FAKE, BIG, None) == code


BAD_EPILOGUES = [(dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(act_begin=-1), INVALID), (dict(act_begin=65), INVALID),
                 (dict(gate_rows=-1), INVALID), (dict(ldy=63), INVALID), (dict(ldr=63, residual=FAR), INVALID),
                 (dict(gate=FAR + 1), ALIGN), (dict(residual=FAR + 1), ALIGN), (dict(residual=FAKE + 2), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_EPILOGUES)
def test_epilogue_refusals(L, kw, code):
    assert L.svdq_fp8_gemm(FAKE, FAKE, layer(), epi(**kw), 16, FAKE, 0, FAKE, BIG, None) == code
    assert L.svdq_fp8_linear(FAKE, layer(), epi(**kw), 16, FAKE, 0, FAKE, BIG, None) == code


def test_product_refusals(L):
    for args, code in [((None, FAKE, layer(), None, 16, FAKE, 0), INVALID), ((FAKE + 8, FAKE, layer(), None, 16, FAKE, 0), ALIGN),
                       ((FAKE, None, layer(), None, 16, FAKE, 0), INVALID), ((FAKE, FAKE, None, None, 16, FAKE, 0), INVALID),
                       ((FAKE, FAKE, layer(), None, -1, FAKE, 0), INVALID),
                       ((FAKE, FAKE, layer(), None, B.SVDQ_MAX_DIM + 1, FAKE, 0), UNSUPPORTED),
                       ((FAKE, FAKE, layer(), None, 16, None, 0), INVALID), ((FAKE, FAKE, layer(), None, 16, FAKE, 2), INVALID),
                       ((FAKE, FAKE, layer(), None, 16, FAKE + 2, 1), ALIGN)]:
        assert L.svdq_fp8_gemm(*args, FAKE, BIG, None) == code, args
    assert L.svdq_fp8_gemm(FAKE, FAKE, layer(), None, 0, None, 0, None, 0, None) == B.SVDQ_OK  # nothing to do
    need = L.svdq_fp8_linear_workspace_size(16, 200, 64)
    assert need >= 2 * 16 * 129
    for args, code in [((None, layer(), None, 16, FAKE, 0, FAKE, BIG), INVALID), ((FAKE + 1, layer(), None, 16, FAKE, 0, FAKE, BIG), ALIGN),
                       ((FAKE, layer(), None, 16, FAKE, 0, None, 0), WS), ((FAKE, layer(), None, 16, FAKE, 0, FAKE, need - 1), WS),
                       ((FAKE, layer(), None, 16, FAKE, 0, FAKE + 16, BIG), ALIGN)]:
        assert L.svdq_fp8_linear(*args, None) == code, args
    assert L.svdq_fp8_linear(None, layer(), None, 0, None, 0, None, 0, None) == B.SVDQ_OK


def test_grouped_refusals(L):
    for args, code in [((FAKE, FAKE, 16, None, None, grouped(), None, 16, FAKE, 0), INVALID),
                       ((FAKE, FAKE, 16, None, FAKE + 2, grouped(), None, 16, FAKE, 0), ALIGN),
                       ((FAKE, FAKE, 16, FAKE + 1, FAKE, grouped(), None, 16, FAKE, 0), ALIGN),
                       ((FAKE, FAKE, 15, None, FAKE, grouped(), None, 16, FAKE, 0), INVALID),
                       ((FAKE, FAKE, 0, FAKE, FAKE, grouped(), None, 16, FAKE, 0), INVALID),
                       ((FAKE, FAKE, B.SVDQ_MAX_DIM + 1, FAKE, FAKE, grouped(), None, 16, FAKE, 0), UNSUPPORTED),
                       ((FAKE, FAKE, 16, None, FAKE, None, None, 16, FAKE, 0), INVALID),
                       ((FAKE, FAKE, 16, None, FAKE, grouped(experts=0), None, 16, FAKE, 0), INVALID),
                       ((FAKE, FAKE, 16, None, FAKE, grouped(experts=1025), None, 16, FAKE, 0), UNSUPPORTED),
                       ((FAKE, FAKE, 16, None, FAKE, grouped(), epi(gate=FAR), 16, FAKE, 0), UNSUPPORTED),
                       ((FAKE, FAKE, 16, None, FAKE, grouped(), epi(residual=FAR), 16, FAKE, 0), UNSUPPORTED),
                       ((FAKE, FAKE, 16, None, FAKE, grouped(), epi(act=9), 16, FAKE, 0), INVALID),
                       ((None, FAKE, 16, None, FAKE, grouped(), None, 16, FAKE, 0), INVALID),
                       ((FAKE, None, 16, None, FAKE, grouped(), None, 16, FAKE, 0), INVALID),
                       ((FAKE, FAKE, 16, None, FAKE, grouped(), None, 16, None, 0), INVALID)]:
        assert L.svdq_fp8_grouped_gemm(*args, None) == code, args
    assert L.svdq_fp8_grouped_gemm(None, None, 0, None, None, grouped(), None, 0, None, 0, None) == B.SVDQ_OK
    need = L.svdq_fp8_grouped_linear_workspace_size(16, 9, 4, 200, 64)
    assert need >= 2 * 9 * 129
    ok = (FAKE, 9, FAKE, FAKE, grouped(), None, 16, FAKE, 0)
    assert L.svdq_fp8_grouped_linear(*ok, None, 0, None) == WS
    assert L.svdq_fp8_grouped_linear(*ok, FAKE, need - 1, None) == WS
    assert L.svdq_fp8_grouped_linear(None, *ok[1:], FAKE, need, None) == INVALID
    assert L.svdq_fp8_grouped_linear(FAKE + 1, *ok[1:], FAKE, need, None) == ALIGN


def test_quantizer_refusals(L):
    for args, code in [((None, 4, 200, FAKE, FAKE), INVALID), ((FAKE + 1, 4, 200, FAKE, FAKE), ALIGN), ((FAKE, 4, 0, FAKE, FAKE), INVALID),
                       ((FAKE, -1, 200, FAKE, FAKE), INVALID), ((FAKE, 4, 200, None, FAKE), INVALID), ((FAKE, 4, 200, FAKE + 4, FAKE), ALIGN),
                       ((FAKE, 4, 200, FAKE, None), INVALID), ((FAKE, 4, B.SVDQ_MAX_DIM + 1, FAKE, FAKE), UNSUPPORTED),
                       ((FAKE, B.SVDQ_MAX_DIM, B.SVDQ_MAX_DIM, FAKE, FAKE), UNSUPPORTED)]:
        assert L.svdq_fp8_quantize_act(*args, None) == code, args
    assert L.svdq_fp8_quantize_act(None, 0, 200, None, None, None) == B.SVDQ_OK
    for args, code in [((None, 0, 1, 9, 9, 0, FAKE, FAKE), INVALID), ((FAKE, 2, 1, 9, 9, 0, FAKE, FAKE), INVALID),
                       ((FAKE + 1, 0, 1, 9, 9, 0, FAKE, FAKE), ALIGN), ((FAKE + 2, 1, 1, 9, 9, 0, FAKE, FAKE), ALIGN),
                       ((FAKE, 0, 0, 9, 9, 0, FAKE, FAKE), INVALID), ((FAKE, 0, 1, 0, 9, 0, FAKE, FAKE), INVALID),
                       ((FAKE, 0, 1, 9, 9, 0, None, FAKE), INVALID), ((FAKE, 0, 1, 9, 9, 0, FAKE + 8, FAKE), ALIGN),
                       ((FAKE, 0, 1, 9, 9, 0, FAKE, None), INVALID),
                       ((FAKE, 0, 1, B.SVDQ_MAX_DIM, B.SVDQ_MAX_DIM, 0, FAKE, FAKE), UNSUPPORTED),
                       ((FAKE, 0, 1 << 20, 1000, 1000, 0, FAKE, FAKE), UNSUPPORTED)]:
        assert L.svdq_fp8_quantize_weights(*args, None) == code, args


def test_workspace_sizes(L):
    assert L.svdq_fp8_gemm_workspace_size(0, 64, 64) == 0 and L.svdq_fp8_gemm_workspace_size(4, 0, 64) == 0
    assert L.svdq_fp8_linear_workspace_size(0, 64, 64) == 0 and L.svdq_fp8_linear_workspace_size(4, 64, B.SVDQ_MAX_DIM + 1) == 0
    for b, m, n in ((1, 1, 1), (5, 129, 70), (4096, 1152, 4608), (4194304, 128, 128)):
        G = -(-m // 128)
        assert L.svdq_fp8_linear_workspace_size(b, m, n) >= G * b * 129 + L.svdq_fp8_gemm_workspace_size(b, n, m)
        assert L.svdq_fp8_grouped_linear_workspace_size(2 * b if b < 1 << 21 else b, b, 8, m, n) >= G * b * 129
    assert L.svdq_fp8_grouped_linear_workspace_size(4, 4, 1025, 64, 64) == 0
    assert L.svdq_sort_rows_workspace_size(0, 1, 1) == 0 and L.svdq_sort_rows_workspace_size(32, 4, 64) == 0
    assert L.svdq_sort_rows_workspace_size(1 << 20, 4, 1024) <= 256 * 1025 * 4
    assert L.svdq_sort_rows_workspace_size(1 << 21, 4, 64) == 0  # too many slots


def test_sort_refusals(L):
    ok = dict(expert=FAKE, t=8, k=2, experts=4, off=FAR, row=FAR2, index=FAR2 + 4096, ws=None, size=0)

    def call(**kw):
        d = dict(ok, **kw)
        return L.svdq_sort_rows(d["expert"], d["t"], d["k"], d["experts"], d["off"], d["row"], d["index"], d["ws"], d["size"], None)

    for kw, code in [(dict(expert=None), INVALID), (dict(off=None), INVALID), (dict(row=None), INVALID), (dict(index=None), INVALID),
                     (dict(t=-1), INVALID), (dict(k=0), INVALID), (dict(k=1025), UNSUPPORTED), (dict(experts=0), INVALID),
                     (dict(experts=1025), UNSUPPORTED), (dict(t=B.SVDQ_MAX_DIM, k=2), UNSUPPORTED), (dict(expert=FAKE + 2), ALIGN),
                     (dict(off=FAR + 1), ALIGN), (dict(row=FAR2 + 2), ALIGN), (dict(index=FAR2 + 4097), ALIGN),
                     (dict(row=FAKE), INVALID), (dict(index=FAKE + 60), INVALID), (dict(index=FAR2 + 60), INVALID),
                     (dict(off=FAR2 + 4096 + 60), INVALID), (dict(t=4000), WS)]:
        assert call(**kw) == code, kw
        assert L.svdq_last_error()
    need = L.svdq_sort_rows_workspace_size(4000, 2, 4)
    apart = dict(t=4000, index=FAR2 + (1 << 20))
    assert need == 2 * 5 * 4
    assert call(**apart, ws=FAR + (1 << 20), size=need - 1) == WS and call(**apart, ws=FAR + 8, size=need) == ALIGN
    assert call(**apart, ws=FAKE + 16, size=need) == INVALID


def test_scatter_refusals(L):
    ok = dict(x=FAKE, t=8, n=32, dtype=0, index=FAR, weight=None, k=2, rows=FAR2, R=16, drows=FAR2 + (1 << 20), dw=FAR + 4096)

    def grad(**kw):
        d = dict(ok, **kw)
        return L.svdq_combine_rows_grad(d["x"], d["t"], d["n"], d["dtype"], d["index"], d["weight"], d["k"], d["rows"], d["R"],
                                        d["drows"], d["dw"], None)

    def dispatch(**kw):
        d = dict(ok, **kw)
        return L.svdq_dispatch_rows(d["x"], d["t"], d["n"], d["dtype"], d["index"], d["weight"], d["k"], d["R"], d["drows"], None)

    for kw, code in [(dict(x=None), INVALID), (dict(t=-1), INVALID), (dict(n=0), INVALID), (dict(R=-1), INVALID), (dict(dtype=2), INVALID),
                     (dict(index=None), INVALID), (dict(k=0), INVALID), (dict(k=1025), UNSUPPORTED), (dict(n=B.SVDQ_MAX_DIM + 1), UNSUPPORTED),
                     (dict(R=B.SVDQ_MAX_DIM + 1), UNSUPPORTED), (dict(t=B.SVDQ_MAX_DIM + 1), UNSUPPORTED), (dict(x=FAKE + 1), ALIGN),
                     (dict(x=FAKE + 2, dtype=1), ALIGN), (dict(index=FAR + 2), ALIGN), (dict(weight=FAR + 2), ALIGN),
                     (dict(drows=FAR2 + 1), ALIGN), (dict(drows=FAKE), INVALID), (dict(drows=FAKE + 64), INVALID), (dict(drows=FAR), INVALID)]:
        assert grad(**kw) == code, kw
        assert dispatch(**kw) == code, kw
    for kw, code in [(dict(rows=None), INVALID), (dict(rows=FAR2 + 1), ALIGN), (dict(dw=FAR + 4097), ALIGN), (dict(dw=FAR2), INVALID),
                     (dict(dw=FAKE), INVALID), (dict(dw=FAR), INVALID), (dict(drows=FAR2 + 64), INVALID),
                     (dict(drows=FAR2, dw=FAR2 + 64), INVALID)]:
        assert grad(**kw) == code, kw
    assert dispatch(drows=None) == INVALID
    # nothing to do
    assert grad(t=0, x=None, index=None) == B.SVDQ_OK and grad(drows=None, dw=None) == B.SVDQ_OK
    assert dispatch(t=0) == B.SVDQ_OK and dispatch(R=0, drows=None) == B.SVDQ_OK


def test_binding_refuses_tensors_off_the_gpu():
    import torch
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: S.svdq_fp8_quantize_act(x), lambda: S.svdq_fp8_quantize_weights(x), lambda: S.DeviceLayerFp8(x),
                 lambda: S.GroupedDeviceLayerFp8(x.view(1, 4, 128)), lambda: S.svdq_sort_rows(i, 4), lambda: S.svdq_dispatch_rows(x, i),
                 lambda: S.svdq_combine_rows_grad(x, i), lambda: S.DeviceLayerFp8(x[0]), lambda: S.GroupedDeviceLayerFp8(x)):
        with pytest.raises(ValueError):
            call()


def test_reference_quantizer():
    """The reference's codes are the nearest of the 253 finite E4M3 values and its scales the least that hold a block."""
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 3000), rng.uniform(-0.02, 0.02, 3000), F.VALUES[np.isfinite(F.VALUES)]])
    got = F.VALUES[F.encode(v)]
    grid = F.VALUES[np.isfinite(F.VALUES)]
    best = np.abs(v[:, None] - grid[None]).min(1)
    assert np.array_equal(np.abs(got - v), best)
    mid = (F.VALUES[:0x7E] + F.VALUES[1:0x7F]) / 2  # ties go to the even code
    assert (F.encode(mid) % 2 == 0).all()
    for a in (1e-3, 0.875, 0.8750001, 448, 448.0001, 2.0 ** -118 * 1.75, 2.0 ** -119, 0, 3.3e38):
        e = F.exponent(a)
        assert a <= 448 * 2.0 ** e and (e == -126 or a > 448 * 2.0 ** (e - 1)) and e == F._fast_exponent(a)
