"""E4M3 blocks in 64 bits, with numpy: the format's values, scales and nearest codes by
search, and the products that are built from them."""

import numpy as np

G = 128


def values():
    """The values of the codes 0 .. 126."""
    c = np.arange(127)
    e, f = c // 8, c % 8
    return np.where(e > 0, (1.0 + f / 8.0) * 2.0 ** (e - 7.0), f / 8.0 * 2.0**-6)


def decode(codes):
    c = np.asarray(codes).astype(np.int64)
    v = np.append(values(), np.nan)[c & 127]
    return np.where(c > 127, -v, v)


def _blocks(x, rows):
    T, d = x.shape
    R, C = -(-T // rows), -(-d // G)
    p = np.zeros((R * rows, C * G))
    p[:T, :d] = x
    return p.reshape(R, rows, C, G)


def spread(s, rows, shape):
    """A block's scale [row blocks, groups] for each element."""
    return np.repeat(np.repeat(s, rows, 0)[: shape[0]], G, 1)[:, : shape[1]]


def scales(x, rows, kind):
    """(stored, value) of every block [row blocks, groups]; a block that is not finite: NaN."""
    with np.errstate(invalid="ignore", over="ignore"):
        b = _blocks(np.asarray(x, dtype=np.float64), rows)
        bad = ~np.isfinite(b).all((1, 3))
        amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max((1, 3)))
        if kind == "f32":
            s = np.maximum((amax / 448.0).astype(np.float32), np.float32(2.0**-126))
            s[bad] = np.nan
            return s, s.astype(np.float64)
        e = np.full(amax.shape, -126, dtype=np.int64)
        for k in range(-126, 128):  # the least e that holds amax
            e = np.where(amax > 448.0 * 2.0**k, min(k + 1, 127), e)
        return np.where(bad, 255, e + 127).astype(np.uint8), np.where(bad, np.nan, 2.0**e)


def nearest(q):
    """Codes nearest to q, ties to the even code, by search."""
    t = values()
    y = np.minimum(np.abs(q), 448.0)
    low = np.clip(np.searchsorted(t, y, side="right") - 1, 0, 126)
    high = np.minimum(low + 1, 126)
    up, down = t[high] - y, y - t[low]
    code = np.where((up < down) | ((up == down) & (low % 2 == 1)), high, low)
    return np.where(q < 0, code + 128, code).astype(np.uint8)


def quantize(x, rows, kind):
    """codes, stored scales and scale values; scales of rows as [groups, T]."""
    x = np.asarray(x, dtype=np.float64)
    stored, value = scales(x, rows, kind)
    s = spread(value, rows, x.shape)
    with np.errstate(invalid="ignore"):
        q = np.where(np.isnan(s), 0.0, np.where(np.isfinite(x), x, 0.0) / np.where(np.isnan(s), 1.0, s))
    codes = nearest(q)
    return codes, (stored.T.copy() if rows == 1 else stored), value


def scale_values(stored):
    stored = np.asarray(stored)
    if stored.dtype == np.uint8:
        return np.where(stored == 255, np.nan, 2.0 ** (stored.astype(np.float64) - 127.0))
    return stored.astype(np.float64)


def dequantize(codes, stored, rows):
    s = scale_values(stored)
    return decode(codes) * spread(s.T if rows == 1 else s, rows, codes.shape)


def _tops(codes, stored, rows):
    """For every 8 adjacent elements the power of two of the largest (subnormals and zeros: 2^-6), times the scale."""
    T, d = codes.shape
    v = np.abs(decode(codes))
    with np.errstate(divide="ignore"):
        e = np.where(v >= 2.0**-6, np.exp2(np.floor(np.log2(np.maximum(v, 2.0**-6)))), 2.0**-6)
    e = np.pad(e, ((0, 0), (0, -d % 8))).reshape(T, -1, 8).max(2)
    s = scale_values(stored)
    return e * spread(s.T if rows == 1 else s, rows, codes.shape)[:, ::8]


def linear(xq, xs, W, ws):
    """The product, the sum of its terms' magnitudes, and the sum over 8 adjacent terms each of the largest's power of two."""
    x, w = dequantize(xq, xs, 1), dequantize(W, ws, G)
    return x @ w.T, np.abs(x) @ np.abs(w).T, _tops(xq, xs, 1) @ _tops(W, ws, G).T


# The 8-bit matrix instructions add the products of 8 adjacent elements at a fixed point: with the largest
# exponents e and f of two factors that meet, what lies below 2^(e + f - 13) of each product is cut off (measured with
# exact powers: 2^16 + 2^3 is kept, 2^16 + 2^2 gives 2^16; across the eights the sums are fp32's).  So each of the 8
# products loses less than 2^-13 of that power of two.  Beyond that a block's inner sum and the sum over the blocks
# are fp32 additions in some order: each loses at most a step (2^-23) of a partial sum that is at most the sum of the
# magnitudes; the factor sx sw and its product are two roundings more.  Then the result is rounded to its type once.
def linear_bound(ref, mag, tops, k, out):
    groups = -(-k // G)
    b = (k + groups + 4) * 2.0**-23 * mag + 8 * 2.0**-13 * tops
    return b + (2.0**-8 * np.abs(ref) + 2.0**-133 if out == "bf16" else 2.0**-24 * np.abs(ref)) * 1.01
