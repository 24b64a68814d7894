"""8-bit floating point with a scale for every block of 128, and dropout by
numbers from a counter, in 64 bits from their definitions.

Plain numpy, for tests only: values come from tables of every code, rounding
from a search for the nearest one, random words from Python integers.
"""

import numpy as np

BLOCK = 128


def table(fmt):
    """The value of each of the 256 codes; NaN and infinities as such."""
    exp_bits, bias = (4, 7) if fmt == "e4m3" else (5, 15)
    man_bits = 7 - exp_bits
    out = np.empty(256)
    for code in range(256):
        sign = -1.0 if code & 0x80 else 1.0
        e, m = (code & 0x7F) >> man_bits, code & ((1 << man_bits) - 1)
        if fmt == "e4m3" and e == 15 and m == 7:
            out[code] = np.nan
        elif fmt == "e5m2" and e == 31:
            out[code] = np.nan if m else sign * np.inf
        elif e == 0:
            out[code] = sign * m * 2.0 ** (1 - bias - man_bits)
        else:
            out[code] = sign * (2 ** man_bits + m) * 2.0 ** (e - bias - man_bits)
    return out


def largest(fmt):
    return 448.0 if fmt == "e4m3" else 57344.0


def nearest(x, fmt):
    """Codes of the values nearest to x, ties to the even code; |x| at most the
    largest value.  The sign of a zero is kept."""
    values = table(fmt)[: 0x7F if fmt == "e4m3" else 0x7C]  # 0, 1, 2, ... ascending
    mag = np.abs(x)
    hi = np.clip(np.searchsorted(values, mag), 1, len(values) - 1)
    lo = hi - 1
    up, down = values[hi] - mag, mag - values[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def exponent(peak, fmt):
    """The least e >= -127 with peak 2^-e at most the largest value; 0 for 0."""
    if peak == 0.0:
        return 0
    e = -127
    while peak * 2.0 ** -e > largest(fmt):
        e += 1
    return e


def quantize(x, fmt="e4m3", rows=1):
    """(codes, scale bytes [blocks of a row, rows of x]) of a float64 matrix in
    blocks of ``rows`` x 128."""
    h, w = x.shape
    codes = np.zeros((h, w), np.uint8)
    blocks = -(-w // BLOCK)
    scale = np.zeros((blocks, h), np.uint8)
    for j in range(blocks):
        for i in range(0, h, rows):
            part = x[i:i + rows, j * BLOCK:(j + 1) * BLOCK]
            if not np.isfinite(part).all():
                codes[i:i + rows, j * BLOCK:(j + 1) * BLOCK] = 0x7F
                scale[j, i:i + rows] = 127
                continue
            e = exponent(np.abs(part).max(), fmt)
            codes[i:i + rows, j * BLOCK:(j + 1) * BLOCK] = nearest(part * 2.0 ** -e, fmt)
            scale[j, i:i + rows] = e + 127
    return codes, scale


def values(codes, scale, fmt="e4m3"):
    """What codes and scale bytes stand for, in float64."""
    w = codes.shape[1]
    unit = np.ldexp(1.0, scale.T.astype(np.int64) - 127).repeat(BLOCK, axis=1)[:, :w]
    return table(fmt)[codes] * unit


def philox(counter, key):
    """The four words of Philox4x32-10 for a counter of four words and a key of two."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep(T, n, p, seed, offset=0, row0=0):
    """Truth values [T, n]: which elements a dropout keeps."""
    out = np.empty((T, -(-n // 4) * 4), bool)
    border = round(p * 2 ** 32)
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    key = seed & 0xFFFFFFFF, seed >> 32
    for t in range(T):
        for q in range(out.shape[1] // 4):
            out[t, 4 * q:4 * q + 4] = [w >= border for w in
                                       philox((q, row0 + t, offset & 0xFFFFFFFF, offset >> 32), key)]
    return out[:, :n]


def drop(x, kept, p):
    """The kept elements times 1 / (1 - p) in fp32, rounded to fp32; the others 0."""
    grow = np.float32(1.0 / (1.0 - p))
    with np.errstate(invalid="ignore", over="ignore"):
        return np.where(kept, (x.astype(np.float32) * grow).astype(np.float64), 0.0)
