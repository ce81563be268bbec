"""Newton-Schulz orthogonalisation and the Muon step in 64 bits, and in the fp16 parts that the
kernels hold, which say how far off they may be."""
from __future__ import annotations

import numpy as np

from .layernorm_oracle import HALF_ULP, rounding

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def start(u, eps):
    return u / (np.linalg.norm(u) + eps)


def orthogonalize(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    a, b, c = coefficients
    x = start(np.asarray(u, np.float64), eps)
    x = x.T if x.shape[0] > x.shape[1] else x
    for _ in range(steps):
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.T if u.shape[0] > u.shape[1] else x


def momentum(g, m, mu, nesterov=True):
    """(new momentum, update)"""
    m = mu * m + (1 - mu) * g
    return m, (1 - mu) * g + mu * m if nesterov else m


def step(w, g, m, lr, mu, wd, scale, nesterov=True, **ns):
    m, u = momentum(g, m, mu, nesterov)
    return w * (1 - lr * wd) - lr * scale * orthogonalize(u, **ns), m


def parts(v, scale):
    """v as two fp16 parts under a power of two, as they stand for values."""
    v = (np.asarray(v, np.float32) * np.float32(scale)).astype(np.float32)
    hi = v.astype(np.float16).astype(np.float32)
    return hi / np.float32(scale), (v - hi).astype(np.float16).astype(np.float32) / np.float32(scale)


def in_parts(u, dtype, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """The iteration in the kernels' formats: X in two fp16 parts under 2^12, A and B off their
    diagonals under 2^8, products of the upper parts (bf16 results) or of both, in fp32."""
    a, b, c = coefficients
    x = start(np.asarray(u, np.float64), eps)
    x = x.T if x.shape[0] > x.shape[1] else x
    half = dtype == "bf16"

    def product(p, q):
        return p[0] @ q[0] if half else p[1] @ q[0] + p[0] @ q[1] + p[0] @ q[0]

    def held(v):
        d = np.diag(v).copy()
        return d, parts(v - np.diag(d), 256.0)

    for k in range(steps):
        x = parts(x, 4096.0)
        d, o = held(product(x, (x[0].T, x[1].T)))
        off = o[0] if half else o[0] + o[1]
        q = b * (off + np.diag(d)) + c * (product(o, o) + (d[:, None] + d[None, :]) * off + np.diag(d * d))
        d, o = held(q.astype(np.float32))
        x = (np.float32(a) + d[:, None]) * (x[0] + x[1]) + product(o, x)
    return x.T if u.shape[0] > u.shape[1] else x


def bounds(u, true, dtype, **ns):
    """How far a result may be off before it is rounded, as (its 2-norm, its largest value). The
    kernels round where in_parts does and differ by the order of their fp32 sums alone: twice
    and four times as far off as that is, and no nearer asked than five steps' roundings of what
    is carried (2^-22 of the norm, which a step takes up to 3.5 times further; products of upper
    parts 2^-11)."""
    off = np.abs(in_parts(u, dtype, **ns) - true)
    least = (2.0 ** -11 if dtype == "bf16" else 2.0 ** -19) * np.linalg.norm(true)
    return 2 * np.linalg.norm(off) + least, 4 * off.max() + 4 * least / np.sqrt(true.size)


__all__ = ["HALF_ULP", "rounding", "orthogonalize", "step", "in_parts", "bounds", "momentum"]
