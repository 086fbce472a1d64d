"""64-bit references of the products with an epilogue, with the error bounds
their 32-bit computation allows.  Numpy only; nothing of the library.

Bounds (u = 2^-24, the unit roundoff of fp32; S the sum of the magnitudes of the
terms of v):
  * v: the isum * sx products are exact, each group's FMA and each addition of the
    low-rank product rounds once (MFMA additions may truncate: 2 u), as do the
    addition of the bias, the reduction of at most 16 partial sums and, in the
    8-bit setting, the conversion and the scaling:
    |dv| <= (G + rank + 24) 2 u S.
  * activations: their derivative is at most 1.13, so dv passes with that factor;
    their own error is below.  exp(x) is 2^fl(x log2 e): relative error
    |x| 4 u (argument: its own rounding and the constants') + 4 u (v_exp, v_rcp
    and the multiplications, an ulp each).
  * gate: one multiplication; residual: one addition; then the output's rounding.
"""
import math

import numpy as np

U = 2.0 ** -24
GROUP = 64


def bf16(a):
    """Values rounded to bf16 (nearest, ties to even), as float64."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32)
    return (r << 16).astype(np.uint32).view(np.float32).astype(np.float64).reshape(np.shape(a))


def bf16_bits(a):
    """Bits of values that are bf16 values."""
    return (np.ascontiguousarray(a, np.float32).view(np.uint32) >> 16).astype(np.uint16).reshape(np.shape(a))


def act(v, kind):
    """(act(v), the 32-bit evaluation's own error)."""
    a = np.abs(v)
    if kind == "gelu_tanh":
        u2 = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        with np.errstate(over="ignore"):
            y = v / (1 + np.exp(-u2))
        # 2u: three roundings in its polynomial, then exp's; the sigmoid passes on the share 1 / (1 + e^2u)
        return y, np.abs(y) * (np.abs(u2) * 8 + 8) * U + 1e-30
    if kind == "gelu_erf":
        from scipy.special import erfc
        phi = 0.5 * erfc(-v / math.sqrt(2))
        h = 0.5 * erfc(a / math.sqrt(2))
        # Abramowitz and Stegun 7.1.26: 1.5e-7 in erf; h: exp(-x^2) and five steps of the polynomial, whose terms
        # alternate and sum to at most 3 times its value in magnitude
        return v * phi, a * (0.75e-7 + h * (a * a * 4 + 40) * U + 2 * U) + 1e-30
    if kind == "silu":
        with np.errstate(over="ignore"):
            y = v / (1 + np.exp(-v))
        return y, np.abs(y) * (a * 4 + 8) * U + 1e-30
    if kind == "relu":
        return np.maximum(v, 0), np.zeros_like(v)
    return v, np.zeros_like(v)


def epilogue(v, dv, kind="none", act_begin=0, gate=None, gate_rows=None, residual=None, out="f32"):
    """(y before its rounding, bound on |the library's y - it|).  gate, residual: float64 values."""
    y, err = v.copy(), dv.copy()
    ya, ea = act(v[:, act_begin:], kind)
    y[:, act_begin:] = ya
    err[:, act_begin:] = 1.13 * dv[:, act_begin:] + ea
    if gate is not None:
        g = gate[np.arange(v.shape[0]) // (gate_rows or max(v.shape[0], 1))]
        y, err = y * g, err * np.abs(g)
        err = err + np.abs(y) * U
    if residual is not None:
        y = residual + y
        err = err + (np.abs(y) + err) * U
    half = 2.0 ** -8 if out == "bf16" else U  # half a step of the output's type
    return y, err * 1.01 + (np.abs(y) + err) * half * 1.01 + 1e-38


def product_int4(cx, sx, cw, sw, z=None, l2=None, bias=None):
    """cx [b][m], sx [m/64][b], cw [n][m], sw [m/64][n], z [b][r], l2 [n][r], bias [n] -> (v, dv)."""
    b, m = cx.shape
    G = m // GROUP
    v = np.zeros((b, cw.shape[0]))
    S = np.zeros_like(v)
    for g in range(G):
        s = slice(GROUP * g, GROUP * (g + 1))
        t = (cx[:, s].astype(np.float64) @ cw[:, s].T.astype(np.float64)) * np.outer(sx[g], sw[g])
        v += t
        S += np.abs(t)
    return _branch(v, S, G, z, l2, bias)


def product_values(x, w, terms, z=None, l2=None, bias=None):
    """Dequantized operands [b][m], [n][m]; `terms` additions of 32-bit sums."""
    return _branch(x @ w.T, np.abs(x) @ np.abs(w).T, terms, z, l2, bias)


def _branch(v, S, G, z, l2, bias):
    rank = 0
    if z is not None and z.shape[1]:
        rank = z.shape[1]
        zb = bf16(z)
        v, S = v + zb @ l2.T, S + np.abs(zb) @ np.abs(l2).T
    if bias is not None:
        v, S = v + bias, S + np.abs(bias)
    return v, (G + rank + 24) * 2 * U * S


def quantize(x, inv):
    """Rows of bf16 values: (x~ float64 [b][m], codes int8 [b][m], scales float64 [m/64][b])."""
    with np.errstate(over="ignore", invalid="ignore"):
        xt = bf16((x.astype(np.float32) * inv.astype(np.float32)).astype(np.float32)) if inv is not None else x
        g = xt.astype(np.float32).reshape(x.shape[0], x.shape[1] // GROUP, GROUP)
        a = np.minimum(np.abs(g).max(-1) / np.float32(7), np.float32(65504)).astype(np.float16).astype(np.float32)
        q = np.where(a[..., None] > 0, np.rint(g / np.where(a > 0, a, 1)[..., None]), 0)
    return xt, np.clip(q, -7, 7).reshape(x.shape).astype(np.int8), a.T.astype(np.float64)
