"""Plain AdamW step and its 8-bit state in numpy, written from the formulas of include/tgrad.h.

`step64` is the step in 64 bits. `encode_exact` / `decode` are the 8-bit format in 64-bit
arithmetic on real numbers (a code is a position on the grid of representable values), apart
from the library's way through the bits of an fp32 number. `step32` is the same step with
every operation rounded to fp32, which the stored state follows bit for bit.
"""
from __future__ import annotations

import numpy as np

GROUP = 128
M_BITS, Q_BITS = 3, 4       # mantissa bits of a code of m and of q = sqrt(v)


def step64(w, g, m, v, t, lr, b1, b2, eps, wd, coef=1.0):
    """(w before rounding, m, v) after step t."""
    w, g, m, v = (np.asarray(x, np.float64) for x in (w, g, m, v))
    g = g * coef
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    w = w * (1 - lr * wd) - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return w, m, v


def step32(g, m, v, b1, b2, coef=1.0):
    """(m, v) with every operation rounded to fp32."""
    f = np.float32
    g = np.asarray(g, f) * f(coef)
    m = f(b1) * np.asarray(m, f) + f(1 - b1) * g
    v = f(b2) * np.asarray(v, f) + f(1 - b2) * (g * g)
    return m, v


def norm_and_coefficient(grads, max_norm, scale):
    s = sum(float((np.abs(np.asarray(g, np.complex128 if np.iscomplexobj(g) else np.float64)) ** 2).sum())
            for g in grads)
    norm = np.sqrt(s) * scale
    return norm, scale * min(1.0, max_norm / norm) if norm > 0 else scale


def random_bits(seed, t, places):
    """The 32 random bits of each place of the flat state at step t."""
    M = (1 << 64) - 1
    z = (seed + t * 0x9E3779B97F4A7C15) & M
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & M
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & M
    key = (z ^ (z >> 31)) & 0xFFFFFFFF
    with np.errstate(over="ignore"):
        h = np.asarray(places, np.uint64).astype(np.uint32) ^ np.uint32(key)
        h = h * np.uint32(0xBF58476D)
        h = h ^ (h >> np.uint32(16))
        h = h * np.uint32(0x94D049BB)
        return h ^ (h >> np.uint32(13))


def padded(x):
    n = -(-x.size // GROUP) * GROUP
    out = np.zeros(n, x.dtype)
    out[:x.size] = x
    return out


def fields(x):
    """The exponent field, as fp32, of each group's largest magnitude."""
    top = np.abs(x).reshape(-1, GROUP).max(1).astype(np.float32)
    return (top.view(np.uint32) >> 23).astype(np.uint8)


def unit_and_position(x, f, bits):
    """|x| in units of the spacing of its binade's codes, and that spacing. Below the least
    normal code the spacing stays."""
    f = np.repeat(f.astype(np.int64), GROUP)
    a = np.abs(np.asarray(x, np.float64))
    e = np.maximum(np.frexp(np.where(a > 0, a, 1e-300))[1] - 1, -126 + f - 14)
    unit = np.ldexp(1.0, e - bits)
    return unit, a / unit


def encode_exact(x, f, bits, low, low_bits):
    """The magnitudes' codes' values, rounded up where the cut-off part plus low / 2^low_bits
    reaches one."""
    unit, pos = unit_and_position(x, f, bits)
    return np.floor(pos + low.astype(np.float64) / (1 << low_bits)) * unit


def least(f, bits):
    return np.repeat(np.ldexp(1.0, f.astype(np.int64) - 14 - 126 - bits), GROUP)


def decode(code, f, bits):
    """Values of codes without their sign."""
    code, f = code.astype(np.int64), np.repeat(f.astype(np.int64), GROUP)
    e, frac = code >> bits, (code & ((1 << bits) - 1)) / (1 << bits)
    val = np.ldexp(np.where(e > 0, 1 + frac, frac), np.maximum(e, 1) - 127 + f - 14)
    return np.where(f == 255, np.nan, val)


def decode_m(code, f):
    return decode(code & 127, f, M_BITS) * np.where(code >= 128, -1.0, 1.0)


def decode_q(code, f):
    return decode(code, f, Q_BITS)
