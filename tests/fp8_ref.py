"""64-bit reference of the 8-bit floating-point setting: E4M3 codes, one power of
two for each block of 128.  Numpy only; nothing of the library.

Bound of a product (tests/epi_ref.py gives the epilogue's): the products of codes
and the scalings by powers of two are exact; the sum of m products takes at most
m additions, and the sums of a few pieces and the bias at most 24 more, each off
by 2 u (additions of the matrix instruction may truncate) of S, the sum of the
magnitudes:  |dv| <= (m + 24) 2 u S,  which product_values(x, w, m) of epi_ref
states.

bf16 outputs of many rows (tiles): v_mfma_scale_f32_16x16x128_f8f6f4 adds the
products of eight neighbouring channels at the exponent of the largest and keeps 13
bits below it (measured on gfx950: beside a product of 2^16 one of 2^3 survives, one
of 2^2 does not; sums of such eights keep 23).  A product's exponent is that of its
factors', and a factor below E4M3's normal numbers counts as 2^-6.  With
p = max(|x|, 2^(ex-6)) max(|w|, 2^(ew-6)), each of the eight products is off by at
most 2^-13 of the largest p, so v by at most  8 2^-13 sum_eights max p  more, which
aligned(...) returns.
"""
import numpy as np

BLOCK = 128
NAN = 0x7F


def _table():
    byte = np.arange(256)
    ex, man = (byte >> 3) & 15, byte & 7
    v = np.where(ex > 0, (1 + man / 8) * 2.0 ** (ex - 7.0), man * 2.0 ** -9)
    v = np.where(byte & 0x80, -v, v)
    v[0x7F] = v[0xFF] = np.nan
    return v


VALUES = _table()


def encode(v):
    """Bytes of finite values of magnitude <= 448, nearest, ties to the even code: by the two neighbours in the table."""
    grid = VALUES[:0x7F]
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up = (grid[hi] - a < a - grid[lo]) | ((grid[hi] - a == a - grid[lo]) & (hi % 2 == 0))
    code = np.where((hi == 0) | up, hi, lo)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def exponent(a):
    """The least e >= -126 with a <= 448 2^e."""
    e = -126
    with np.errstate(over="ignore"):
        while a > 448 * 2.0 ** e:
            e += 1
    return e


def quantize(v, by):
    """Rows [R][c] in blocks of by x 128: (codes uint8 [R][c], exponents int [R / by][G], the values they stand for)."""
    v = np.asarray(v, np.float64)
    R, c = v.shape
    G, NR = -(-c // BLOCK), -(-R // by)
    codes, es, val = np.zeros((R, c), np.uint8), np.zeros((NR, G), int), np.zeros((R, c))
    for i in range(NR):
        for g in range(G):
            s = (slice(by * i, by * (i + 1)), slice(BLOCK * g, BLOCK * (g + 1)))
            t = v[s]
            if not np.isfinite(t).all():
                codes[s], es[i, g], val[s] = NAN, 0, np.nan
                continue
            e = exponent(np.abs(t).max()) if by > 1 or t.size < 40 else _fast_exponent(np.abs(t).max())
            codes[s] = encode(t * 2.0 ** -e)
            es[i, g] = e
            val[s] = VALUES[codes[s]] * 2.0 ** e
    return codes, es, val


def _fast_exponent(a):
    if a == 0:
        return -126
    f, k = np.frexp(a)
    return max(int(k) - (9 if f <= 0.875 else 8), -126)


def records(codes):
    """Codes [R][c] -> [G][R][128], zero behind the last channel."""
    R, c = codes.shape
    G = -(-c // BLOCK)
    p = np.zeros((R, G * BLOCK), np.uint8)
    p[:, :c] = codes
    return np.ascontiguousarray(p.reshape(R, G, BLOCK).transpose(1, 0, 2))


def aligned(xq, wq, w_by=BLOCK):
    """The additional bound of the 8-bit matrix instruction for quantize()'s results of X [b][m] and W^T [n][m]."""
    def factor(q, by):
        codes, es, val = q
        R, c = val.shape
        e = np.repeat(np.repeat(es, by, 0)[:R], BLOCK, 1)
        p = np.zeros(e.shape)
        p[:, :c] = np.abs(val)
        return np.maximum(p, 2.0 ** (e - 6.0))
    x, w = factor(xq, 1), factor(wq, w_by)
    out = np.zeros((x.shape[0], w.shape[0]))
    for k in range(0, x.shape[1], 8):
        top = np.zeros_like(out)
        for i in range(k, k + 8):
            np.maximum(top, np.outer(x[:, i], w[:, i]), out=top)
        out += top
    return out * 2.0 ** -10
