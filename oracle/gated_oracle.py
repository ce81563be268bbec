"""Gated linear layer and its gradients in 64 bits, and how far the kernels may be off."""
from __future__ import annotations

import numpy as np
from scipy.special import erfc

from .layernorm_oracle import EPS32, HALF_ULP, rounding


def activate(g, act):
    """act(g) and act'(g)."""
    with np.errstate(over="ignore"):
        if act == "relu":
            return np.maximum(g, 0.0), (g > 0).astype(np.float64)
        if act == "gelu":
            cdf = 0.5 * erfc(-g / np.sqrt(2.0))
            return g * cdf, cdf + g * np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)
        p = 1.0 / (1.0 + np.exp(-g))
        return (p, p * (1.0 - p)) if act == "sigmoid" else (g * p, p + g * p * (1.0 - p))


def products(x, wg, wu, bg, bu):
    g, u = x @ wg.T, x @ wu.T
    return g + (0.0 if bg is None else bg), u + (0.0 if bu is None else bu)


def forward(x, wg, wu, bg, bu, act):
    g, u = products(x, wg, wu, bg, bu)
    return activate(g, act)[0] * u


def backward(dy, x, wg, wu, bg, bu, act):
    g, u = products(x, wg, wu, bg, bu)
    a, s = activate(g, act)
    dg, du = dy * u * s, dy * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg.sum(0), du.sum(0)


def gamma(terms, dtype):
    """Relative bound of an fp32 sum of `terms` products in any order, with up to one unit of the
    last place lost in an addition. fp32 factors: six sums, and products of parts that are left
    out, each at most 2^-24 of the whole."""
    if dtype == "f32":
        return (6 * terms + 16) * 2 * EPS32 + 3 * EPS32
    return (terms + 16) * 2 * EPS32


def errors(x, wg, wu, bg, bu, act, dtype):
    """g, u, act(g), act'(g) and bounds of how far those of the kernels are off."""
    g, u = products(x, wg, wu, bg, bu)
    k = x.shape[1]
    eg = gamma(k, dtype) * (np.abs(x) @ np.abs(wg).T + (0.0 if bg is None else np.abs(bg)))
    eu = gamma(k, dtype) * (np.abs(x) @ np.abs(wu).T + (0.0 if bu is None else np.abs(bu)))
    a, s = activate(g, act)
    # the functions: a polynomial to 1e-6, exponentials whose argument is rounded (g^2 / 2 and
    # less, of which a unit is as much of the value), reciprocals and products to a unit each
    own = 0.0 if act == "relu" else 1.2e-6 + (1.0 + g * g) * 4 * EPS32
    # slopes of act and act' are below 1.2 (gelu 1.13 and 0.8, silu 1.1 and 0.5)
    ea = own * np.abs(a) + 1.2 * eg + 1e-37
    es = own * (np.abs(s) + np.abs(g) * np.exp(-np.minimum(0.5 * g * g, 700.0)) + (act != "relu")) + 1.2 * eg
    if act == "relu":   # next to zero either side is right
        es = np.where(np.abs(g) <= eg, 1.0, 0.0)
    return g, u, a, s, eg, eu, ea, es


def forward_bound(x, wg, wu, bg, bu, act, dtype):
    g, u, a, s, eg, eu, ea, es = errors(x, wg, wu, bg, bu, act, dtype)
    e = ea * np.abs(u) + np.abs(a) * eu + ea * eu + 4 * EPS32 * np.abs(a * u)
    return e + rounding(np.abs(a * u) + e, dtype)


def backward_bounds(dy, x, wg, wu, bg, bu, act, dtype):
    g, u, a, s, eg, eu, ea, es = errors(x, wg, wu, bg, bu, act, dtype)
    d = np.abs(dy)
    dg, du = np.abs(dy * u * s), np.abs(dy * a)
    eg = d * (es * (np.abs(u) + eu) + eu * np.abs(s)) + 4 * EPS32 * dg
    eu = d * ea + 4 * EPS32 * du
    rows, hidden = dy.shape
    sums = []
    for v, e in ((dg, eg), (du, eu)):
        t = gamma(rows, "f16") * v.sum(0) + e.sum(0)
        sums.append(t + rounding(v.sum(0) + t, dtype))
    # rounded to the type between the products (fp32: in parts that add up to them)
    if dtype != "f32":
        eg, eu = eg + rounding(dg + eg, dtype), eu + rounding(du + eu, dtype)
    aw, au, ax = np.abs(wg), np.abs(wu), np.abs(x)
    out = []
    for true, err in ((dg @ aw + du @ au, eg @ aw + eu @ au), (dg.T @ ax, eg.T @ ax), (du.T @ ax, eu.T @ ax)):
        terms = 2 * hidden if not out else rows
        e = err + gamma(terms, dtype) * (true + err)
        out.append(e + rounding(true + e, dtype))
    return out + sums


__all__ = ["HALF_ULP", "activate", "forward", "backward", "forward_bound", "backward_bounds"]
