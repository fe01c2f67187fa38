"""AdamW in numpy, written from its formulas: m and v in the kernel's fp32
operation order (IEEE operations, so the values and the 8-bit codes are equal bit
for bit), p in 64 bits with a bound."""

from __future__ import annotations

import numpy as np

BLOCK = 256
F = np.float32


def mix(h):
    h = np.asarray(h, dtype=np.uint32)
    with np.errstate(over="ignore"):
        h = (h ^ (h >> np.uint32(16))) * np.uint32(0x6A09E667)
        h = (h ^ (h >> np.uint32(15))) * np.uint32(0xBB67AE85)
    return h ^ (h >> np.uint32(16))


def noise(seed, step, tensor, n):
    """The 32 random bits of elements 0 .. n - 1."""
    M = 0xFFFFFFFF
    key = mix((int(mix(((seed & M) + step * 0x9E3779B9) & M)) + tensor * 0x510E527F) & M)
    return mix((np.arange(n, dtype=np.uint64) * 0x9E3779B9 + int(key)) & M)


def table(bias):
    """Values of the codes 0 .. 255 of 8-bit floats without a sign, 3 mantissa bits."""
    c = np.arange(256)
    e, f = c >> 3, c & 7
    return np.where(e > 0, (8.0 + f) * 2.0 ** (e - bias - 3.0), f * 2.0 ** (-2.0 - bias))


FORMAT = {"m": (7, 8, 126), "v": (15, 16, 254)}  # bias, exponent of the largest code, largest code


def decode(codes, scales, which):
    bias, _, top = FORMAT[which]
    codes = np.asarray(codes, dtype=np.int64)
    s = np.repeat(2.0 ** (np.asarray(scales, dtype=np.float64) - 127), BLOCK)[: codes.size]
    mag = codes & 127 if which == "m" else codes
    val = np.where(mag > top, np.nan, table(bias)[np.minimum(mag, top)]) * s
    return np.where((codes & 128) > 0, -val, val) if which == "m" else val


def encode(x, rnd16, which):
    """(codes, scales) of fp32 values, by search in the format's table."""
    bias, topexp, top = FORMAT[which]
    x = np.asarray(x, dtype=np.float64)
    n = x.size
    nb = (n + BLOCK - 1) // BLOCK
    pad = np.zeros(nb * BLOCK)
    pad[:n] = np.where(np.isfinite(x), np.abs(x), 0)
    most = pad.reshape(nb, BLOCK).max(1)
    scales = np.empty(nb, dtype=np.int64)
    for b, a in enumerate(most):
        e = 1
        while e < 254 and a >= 1.75 * 2.0**topexp * 2.0 ** (e - 127):
            e += 1
        scales[b] = e
    y = np.where(np.isfinite(x), np.abs(x), 0) / np.repeat(2.0 ** (scales - 127.0), BLOCK)[:n]
    t = table(bias)[: top + 1]
    lo = np.clip(np.searchsorted(t, y, side="right") - 1, 0, top)
    hi = np.minimum(lo + 1, top)
    gap = t[hi] - t[lo]
    share = np.where(gap > 0, (y - t[lo]) / np.where(gap > 0, gap, 1), 0)
    code = np.where(share + rnd16 / 65536.0 >= 1, hi, lo)
    if which == "v":
        code = np.where((x > 0) & (code == 0), 1, code)
    code = np.where(np.isfinite(x), code, top + 1)
    if which == "m":
        code = code + 128 * (x < 0)
    return code.astype(np.uint8), scales.astype(np.uint8)


def step(p, g, m, v, h):
    """One step: (p in 64 bits, bound of |p - p_gpu|, m, v in fp32).  m and v in fp32."""
    p, g, m, v = (np.asarray(t, dtype=F) for t in (p, g, m, v))
    b1, b2 = F(h["beta1"]), F(h["beta2"])
    with np.errstate(all="ignore"):
        gs = g * F(h["grad_scale"])
        m = b1 * m + (F(1) - b1) * gs
        v = b2 * v + (F(1) - b2) * (gs * gs)
        bc1, bc2 = 1 - float(b1) ** h["step"], 1 - float(b2) ** h["step"]
        lr, wd, eps = (float(F(h[k])) for k in ("lr", "weight_decay", "eps"))
        p64 = p.astype(np.float64)
        decay = lr * wd * p64
        move = lr * (m.astype(np.float64) / bc1) / (np.sqrt(v.astype(np.float64) / bc2) + eps)
        new = p64 - decay - move
        # the last subtraction rounds p; the update is a chain of at most 12 operations,
        # each off by at most 2 steps of 2^-23 (the approximate quotient and root)
        bound = 2.0**-24 * np.abs(new) + 24 * 2.0**-23 * (np.abs(decay) + np.abs(move)) + 1e-45
    return new, bound, m, v
