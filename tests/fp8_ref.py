"""64-bit reference of the 8-bit floating-point setting: E4M3 codes, one power of
two for each block of 128.  Numpy only; nothing of the library.

Bound of a product (tests/epi_ref.py gives the epilogue's): the products of codes
and the scalings by powers of two are exact; the sum of m products takes at most
m additions, and the sums of a few pieces and the bias at most 24 more, each off
by 2 u (additions of the matrix instruction may truncate) of S, the sum of the
magnitudes:  |dv| <= (m + 24) 2 u S,  which product_values(x, w, m) of epi_ref
states.
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
