"""Layer norm over the last axis and its gradients in 64 bits, and how far fp32 sums may be off."""
from __future__ import annotations

import numpy as np

EPS32 = 2.0 ** -24
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# absolute half steps below the smallest normal number
SUBNORMAL = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def statistics(x, eps):
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    return mean, rstd


def forward(x, w, b, eps):
    mean, rstd = statistics(x, eps)
    y = (np.asarray(x, np.float64) - mean[..., None]) * rstd[..., None]
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, mean, rstd


def backward(dy, x, w, mean, rstd):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    n = (x - mean) * rstd
    h = dy if w is None else dy * np.asarray(w, np.float64)
    dx = rstd * (h - h.mean(1, keepdims=True) - n * (h * n).mean(1, keepdims=True))
    return dx, (dy * n).sum(0), dy.sum(0)


def gamma(terms):
    """Relative bound of an fp32 sum of `terms` terms in any order: each term meets at most
    `terms` additions and a few roundings of its own."""
    return (terms + 8) * EPS32


def rounding(x, dtype):
    return np.abs(x) * HALF_ULP[dtype] + SUBNORMAL[dtype]


def forward_bounds(x, w, b, eps, dtype, seq):
    """Bounds of (y, mean, rstd), where no value meets more than `seq` additions of a sum."""
    x = np.asarray(x, np.float64)
    y, mean, rstd = forward(x, w, b, eps)
    em = gamma(seq) * np.abs(x).mean(-1)
    d = np.abs(x - mean[..., None])
    # var: the sum's own error, and its terms' from the mean's error and their rounding
    ev = (gamma(seq) * (d ** 2).mean(-1) + 2 * (em + EPS32 * d.mean(-1)) * d.mean(-1) + em ** 2
          + 4 * EPS32 * eps)
    er = rstd * (0.5 * ev * rstd ** 2 + 4 * EPS32)
    n = d * rstd[..., None]
    en = rstd[..., None] * (em[..., None] + 2 * EPS32 * d) + d * er[..., None]
    aw = 1.0 if w is None else np.abs(np.asarray(w, np.float64))
    ab = 0.0 if b is None else np.abs(np.asarray(b, np.float64))
    ey = aw * en + 3 * EPS32 * (aw * n + ab)
    return ey + rounding(np.abs(y) + ey, dtype), em + EPS32 * np.abs(mean), er


def backward_bounds(dy, x, w, mean, rstd, dtype, wdtype, seq, rows_seq):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    dx, dw, db = backward(dy, x, w, mean, rstd)
    r = np.asarray(rstd, np.float64)[:, None]
    n = np.abs(x - np.asarray(mean, np.float64)[:, None]) * r
    h = np.abs(dy if w is None else dy * np.asarray(w, np.float64))
    es = gamma(seq) * h.mean(1, keepdims=True)
    et = gamma(seq) * (h * n).mean(1, keepdims=True)
    t = (h * n).mean(1, keepdims=True)
    ex = r * (es + n * et + 6 * EPS32 * (h + h.mean(1, keepdims=True) + n * t))
    ew = gamma(rows_seq) * (np.abs(dy) * n).sum(0)
    eb = gamma(rows_seq) * np.abs(dy).sum(0)
    return (ex + rounding(np.abs(dx) + ex, dtype), ew + rounding(np.abs(dw) + ew, wdtype),
            eb + rounding(np.abs(db) + eb, wdtype))
