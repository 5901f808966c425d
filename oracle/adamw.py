"""CPU oracle of the AdamW step, fp64 numpy (TEST INFRASTRUCTURE ONLY: imported by tests/, never
by the library): the step itself and the 8-bit form of its moments, from the definitions."""
from __future__ import annotations

import math

import numpy as np

M32 = 0xffffffff
# largest value, exponent of the smallest normal value, signed
M8 = (448.0, -6, True)
V8 = (1.875 * 2.0 ** 16, -14, False)


def step(p, g, m, v, t, lr, decay, betas, eps, coef=1.0):
    """(p, m, v) after the step number t (from 1)."""
    b1, b2 = betas
    g = np.asarray(g, np.float64) * coef
    m = b1 * np.asarray(m, np.float64) + (1 - b1) * g
    v = b2 * np.asarray(v, np.float64) + (1 - b2) * g * g
    p = np.asarray(p, np.float64)
    u = m / (1 - b1 ** t) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p - lr * (u + decay * p), m, v


def mix(x):
    x = np.asarray(x, np.uint64) & np.uint64(M32)
    x = x ^ (x >> np.uint64(16))
    x = x * np.uint64(0x9E3779B1) & np.uint64(M32)
    x = x ^ (x >> np.uint64(15))
    x = x * np.uint64(0x6A09E667) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def random16(seed, t, tensor, elements):
    """The 16 random bits of the first and of the second moment, for the given elements."""
    i = np.asarray(elements, np.uint64)
    key = int(mix(int(mix((seed + 0x9E3779B1 * t) & M32)) ^ tensor))
    hi = (i >> np.uint64(32)) * np.uint64(0x9E3779B1) & np.uint64(M32)
    h = mix((i & np.uint64(M32)) ^ hi ^ np.uint64(key))
    return (h & np.uint64(0xffff)).astype(np.int64), (h >> np.uint64(16)).astype(np.int64)


def scale_exponent(amax, kind):
    """The smallest power of two (down to 2^-127) under which amax fits."""
    if amax == 0:
        return -127
    e = math.floor(math.log2(amax / kind[0])) - 1
    while kind[0] * 2.0 ** e < amax:
        e += 1
    return max(e, -127)


def grid(kind):
    """All values of the format that are not negative, ascending."""
    top, low, _ = kind
    out = [k * 2.0 ** (low - 3) for k in range(8)]
    e = low
    while 2.0 ** e <= top:
        out += [(8 + k) * 2.0 ** (e - 3) for k in range(8)]
        e += 1
    return np.array([x for x in out if x <= top])


def held(values, e, kind, rand16):
    """What each value becomes: the neighbour below (in magnitude) or above it on the grid, above
    with the probability of the fraction between them; e: the exponent of its block's scale."""
    a = np.abs(values) / 2.0 ** e
    g = grid(kind)
    i = np.searchsorted(g, a, side="right") - 1
    lo, hi = g[i], g[np.minimum(i + 1, len(g) - 1)]
    frac = np.where(hi > lo, (a - lo) / np.where(hi > lo, hi - lo, 1), 0)
    q = np.where(frac + rand16 / 65536.0 >= 1.0, hi, lo)
    if not kind[2]:
        q = np.where((q == 0) & (a > 0), g[1], q)
    return np.sign(values) * q * 2.0 ** e


def decode(codes, scales, kind):
    codes = np.asarray(codes, np.int64)
    mag = codes & 0x7f if kind[2] else codes
    exp, frac = mag >> 3, mag & 7
    bias = 1 - kind[1]
    x = np.where(exp == 0, frac * 2.0 ** (kind[1] - 3), (8 + frac) * 2.0 ** (exp - bias - 3.0))
    x = np.where(kind[2] & (codes >= 128), -x, x)
    return x * 2.0 ** (np.repeat(np.asarray(scales, np.float64), 32) - 127)
