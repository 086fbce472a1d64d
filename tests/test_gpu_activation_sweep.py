"""The epilogue's activations over a dense range of 32-bit values, on the GPU,
against 64-bit values and the error that the header promises for GELU_ERF.

v reaches the epilogue exactly: codes and scales are zero, and the low-rank
branch adds v's three bf16 parts (8 bits each, so every partial sum fits 24
bits).  ``act="none"`` returns v itself, which is checked first."""
import math
import sys

import numpy as np
import pytest

from tests import epi_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = R.U


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a4_rank_corrected_amd as S
    S.lib()
    return S


def values():
    rng = np.random.default_rng(11)
    v = np.concatenate([np.linspace(-6.5, 6.5, 30011), rng.uniform(-1, 1, 20000), rng.uniform(-60, 60, 5000),
                        10.0 ** rng.uniform(-9, 1, 10000) * rng.choice([-1, 1], 10000)])
    return v.astype(np.float32)


def parts(v):
    """fp32 [b] -> three bf16 values each, summing to it exactly, as fp32 [b][3]."""
    cut = lambda x: (np.ascontiguousarray(x, np.float32).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    hi = cut(v)
    mid = cut(v - hi)
    lo = v - hi - mid
    assert np.array_equal(cut(lo), lo) and np.array_equal(hi.astype(np.float64) + mid + lo, v.astype(np.float64))
    return np.stack([hi, mid, lo], 1)


def product(S, fmt, v, n, act):
    """act(v[i]) in each of n columns, through the product of the setting."""
    b = len(v)
    z = torch.from_numpy(parts(v)).cuda()
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")
    l2 = torch.ones((n, 3), dtype=torch.bfloat16, device="cuda")
    if fmt == "int4":
        layer = S.DeviceLayer.from_tensors(64, n, 3, u8(1, n, 32), f16(1, n), None, l2)
        return S.svdq_gemm_w4a4_lowrank_up_epi(u8(1, b, 32), f16(1, b), z, layer, act=act, out_dtype=torch.float32)
    if fmt == "w8a8":
        layer = S.DeviceLayer8.from_tensors(64, n, 3, u8(1, n, 64).view(torch.int8), f16(n), None, l2)
        return S.svdq_w8a8_gemm_lowrank_up_epi(u8(1, b, 64).view(torch.int8), f16(b), z, layer, act=act,
                                               out_dtype=torch.float32)
    layer = S.DeviceLayerFp4.from_tensors(64, n, 3, 1.0, 1.0, u8(1, n, 32), u8(1, n, 4), None, l2)
    return S.svdq_fp4_gemm_lowrank_up_epi(u8(1, b, 32), u8(1, b, 4), z, layer, act=act, out_dtype=torch.float32)


def bound(v, act):
    """(act(v) in 64 bits, bound on the library's distance from it)."""
    if act == "gelu_erf":
        from scipy.special import ndtr
        y = v * ndtr(v)
        # the header's 1e-7 in Phi, and the one rounding of the product (results below 2^-126 may count as zero)
        return y, np.abs(v) * 1e-7 + (np.abs(y) + np.abs(v) * 1e-7) * U + 2.0 ** -126
    return R.act(v, act)


@pytest.mark.parametrize("act", ["gelu_erf", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("fmt,rows", [("int4", 64), ("int4", None), ("w8a8", None), ("fp4", 64), ("fp4", None)])
def test_activation_over_all_magnitudes(S, fmt, rows, act):
    """rows = 64: the row kernel, 64 values in each of 60 calls; None: tiles, all values at once."""
    print(f"sweep {fmt} rows={rows} {act}", flush=True)
    sys.stdout.flush()
    v = values()
    pieces = [v] if rows is None else [v[k * 1021:][:64] for k in range(60)]
    for p in pieces:
        same = product(S, fmt, p, 1, "none")
        got = product(S, fmt, p, 5, act)
        torch.cuda.synchronize()
        assert np.array_equal(same.cpu().numpy()[:, 0], p)
        p = p.astype(np.float64)
        want, tol = bound(p, act)
        err = np.abs(got.cpu().numpy().astype(np.float64) - want[:, None]).max(1)
        bad = ~(err <= tol)
        assert not bad.any(), f"{bad.sum()} of {bad.size} values off, worst {np.max(err / tol):.3g} times the bound"


def test_extremes_of_every_setting(S):
    """Zeros, infinities, NaN and huge values: NaN stays NaN; GELU and SiLU of -inf are NaN."""
    print("extremes", flush=True)
    v = np.array([0.0, -0.0, math.inf, -math.inf, math.nan, 3e38, -3e38, 1e-30, -1e-30], np.float32)
    layer_bias = torch.from_numpy(v).bfloat16().cuda()
    n = len(v)
    for b in (2, 130):
        u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
        f16 = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")
        calls = [
            lambda act: S.svdq_gemm_w4a4_lowrank_up_epi(
                u8(1, b, 32), f16(1, b), None,
                S.DeviceLayer.from_tensors(64, n, 0, u8(1, n, 32), f16(1, n), None, None, None, layer_bias), act=act,
                out_dtype=torch.float32),
            lambda act: S.svdq_w8a8_gemm_lowrank_up_epi(
                u8(1, b, 64).view(torch.int8), f16(b), None,
                S.DeviceLayer8.from_tensors(64, n, 0, u8(1, n, 64).view(torch.int8), f16(n), None, None, None, layer_bias),
                act=act, out_dtype=torch.float32),
            lambda act: S.svdq_fp4_gemm_lowrank_up_epi(
                u8(1, b, 32), u8(1, b, 4), None,
                S.DeviceLayerFp4.from_tensors(64, n, 0, 1.0, 1.0, u8(1, n, 32), u8(1, n, 4), None, None, None, layer_bias),
                act=act, out_dtype=torch.float32)]
        for call in calls:
            for act in ("gelu_erf", "gelu_tanh", "silu", "relu"):
                y = call(act).cpu().numpy()
                big = float(layer_bias[5])
                assert (y[:, :2] == 0).all() and (y[:, 2] == math.inf).all() and np.isnan(y[:, 4]).all(), act
                assert ((y[:, 3] == 0) if act == "relu" else np.isnan(y[:, 3])).all(), act
                assert (y[:, 5] == big).all() and (y[:, 6] == 0).all() and (np.abs(y[:, 7:]) <= 1.01e-30).all(), act
