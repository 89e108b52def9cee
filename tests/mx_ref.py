"""Microscaled formats in numpy, from their definitions: blocks of 32 along a row, a
power of two each."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (E - 10) for E in range(1, 16) for m in range(8)
                   if (E, m) != (15, 7)])


def blocks(x):
    """x [rows x n] in float64 as [rows x blocks x 32], filled up with zeros."""
    rows, n = x.shape
    nb = -(-n // 32)
    v = np.zeros((rows, nb * 32))
    v[:, :n] = x
    return v.reshape(rows, nb, 32)


def exponents(x, kind):
    v = np.abs(blocks(x))
    amax = np.where(np.isfinite(v), v, 0).max(2)
    safe = np.where(amax > 0, amax, 1)
    e = np.floor(np.log2(safe)).astype(int)
    # log2 may round up to the next integer
    e -= np.exp2(e.astype(float)) > safe
    if kind == "fp4":
        e = e - 2
    else:
        e = e - 8
        e += safe > 448 * np.exp2(e.astype(float))
    return np.where(amax > 0, np.maximum(e, -127), 0)


def nearest(a, mags):
    """Indices of the nearest magnitude, ties to the even one, the last for larger."""
    mid = (mags[1:] + mags[:-1]) / 2
    up, down = np.searchsorted(mid, a, "right"), np.searchsorted(mid, a, "left")
    return np.where(up % 2 == 0, up, down)


def encode(x, kind):
    """Codes [rows x n] (one an element) and exponents [rows x blocks]."""
    mags, sign = (E2M1, 8) if kind == "fp4" else (E4M3, 128)
    e = exponents(x, kind)
    v = blocks(x) * np.exp2(-e.astype(float))[:, :, None]
    a = np.abs(v)
    c = nearest(np.where(np.isnan(a), 0, a), mags)
    c = np.where(np.isnan(v), 0 if kind == "fp4" else 127, c)
    c = (c + sign * np.signbit(v)).reshape(x.shape[0], -1)[:, :x.shape[1]]
    return c.astype(np.uint8), e


def decode(c, e, kind):
    """Values of one code an element; byte 255 of exponents as e = 128 is NaN."""
    mags, sign = (E2M1, 8) if kind == "fp4" else (E4M3, 128)
    i = (c % sign).astype(int)
    a = np.where(i < len(mags), mags[np.minimum(i, len(mags) - 1)], np.nan)
    v = np.where(c >= sign, -a, a)
    s = np.where(e == 128, np.nan, np.exp2(e.astype(float)))
    return v * np.repeat(s, 32, 1)[:, :c.shape[1]]


def pack4(c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def unpack4(q):
    return np.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)


def pack_exponents(e):
    """Exponents [rows x blocks] as bytes [steps x rows16 x 8]."""
    rows, nb = e.shape
    out = np.full((-(-nb // 8), -(-rows // 16) * 16, 8), 127, np.uint8)
    for b in range(nb):
        out[b // 8, :rows, 2 * (b % 4) + b % 8 // 4] = e[:, b] + 127
    return out


def unpack_exponents(s, rows, nb):
    e = np.zeros((rows, nb), int)
    for b in range(nb):
        e[:, b] = s[b // 8, :rows, 2 * (b % 4) + b % 8 // 4].astype(int) - 127
    return e
