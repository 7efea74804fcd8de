"""Oracle of the layer around the sequence attention (test infrastructure only:
imported by the tests, never by the library or its binding): layer norm and
the gated feed-forward's projections with their gradients.

Plain numpy in float64 from the definitions.  Next to each result stands a
bound of how far an implementation in fp32 (with rows in fp32 or bf16) may be
from it, from the standard model of rounded arithmetic: a sum of n terms in any
order is off by at most n u times the sum of their magnitudes, u = 2^-24; an
output is rounded once to its type.
"""

from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24          # unit roundoff of fp32
UB = 2.0 ** -8          # unit roundoff of bf16: 8 significant bits, to nearest
OUT = {"f32": U, "bf16": UB}


def _rounded(value, off, kind):
    """The bound of a value that is off by `off` before its rounding."""
    return value, off + OUT[kind] * (np.abs(value) + off)


def norm_sum(x, residual, kind):
    """x + residual; an fp32 sum, then the type's rounding."""
    s = x + residual
    return s, 1.0001 * (U + (UB if kind == "bf16" else 0.0)) * np.abs(s)


def norm_stats(x, eps):
    D = x.shape[1]
    mean = x.mean(1, keepdims=True)
    c = x - mean
    var = (c * c).mean(1, keepdims=True)
    return mean, 1.0 / np.sqrt(var + eps)


def norm(x, weight, bias, eps, kind):
    """{"y", "mean", "r"} of the rows x as they are stored."""
    D = x.shape[1]
    mean, r = norm_stats(x, eps)
    em = (D + 2) * U * np.abs(x).mean(1, keepdims=True)             # of the mean
    c = x - mean
    ec = em + 2 * U * np.abs(c)
    ev = (2 * np.abs(c) * ec + ec * ec).mean(1, keepdims=True) + (D + 3) * U * (c * c).mean(1, keepdims=True)
    er = ev / (r ** -2.0) + 4 * U                                   # relative; twice the derivative's
    y = c * r * weight + bias
    ey = np.abs(weight) * r * (ec + np.abs(c) * er) * 1.01 + 3 * U * np.abs(c * r * weight) + 2 * U * np.abs(y)
    return {"y": _rounded(y, ey, kind), "mean": (mean, em + U * np.abs(mean)), "r": (r, 1.01 * er * r)}


def norm_backward(x, dy, weight, eps, dsum, kind):
    """Gradients for statistics that are fp32 roundings of the exact ones."""
    n, D = x.shape
    mean, r = norm_stats(x, eps)
    c = x - mean
    xh = c * r
    exh = r * (2 * U * np.abs(mean) + 2 * U * np.abs(c)) + 4 * U * np.abs(xh)
    dn = dy * weight
    a, b = dn.mean(1, keepdims=True), (dn * xh).mean(1, keepdims=True)
    ea = (D + 3) * U * np.abs(dn).mean(1, keepdims=True)
    eb = (D + 4) * U * np.abs(dn * xh).mean(1, keepdims=True) + (np.abs(dn) * exh).mean(1, keepdims=True)
    dx = (dn - a - xh * b) * r
    edx = r * (ea + np.abs(xh) * eb + np.abs(b) * exh + 8 * U * (np.abs(dn) + np.abs(a) + np.abs(xh * b)))
    if dsum is not None:
        dx = dx + dsum
        edx = edx + U * np.abs(dx)
    dw, db = (dy * xh).sum(0), dy.sum(0)
    edw = (n + 2) * U * np.abs(dy * xh).sum(0) + (np.abs(dy) * exh).sum(0)
    return {"dx": _rounded(dx, 1.01 * edx, kind), "dweight": (dw, 1.01 * edw + U * np.abs(dw)),
            "dbias": (db, 1.01 * (n + 1) * U * np.abs(dy).sum(0) + U * np.abs(db))}


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activation(act, g):
    """(act(g), act'(g)) of "sigmoid", "silu", "gelu"."""
    if act == "gelu":
        cdf = 0.5 * _erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    s = np.exp(-np.logaddexp(0.0, -g))
    return (s, s * (1 - s)) if act == "sigmoid" else (g * s, s + g * s * (1 - s))


def _projections(x, wg, wu, act):
    """Values and bounds of act(g), act'(g) and u.  The derivatives of the three
    activations are within 1.13 of zero, their second ones within 0.8."""
    D = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = ((D + 1) * U * (np.abs(x) @ np.abs(w).T) for w in (wg, wu))
    a, da = activation(act, g)
    return (a, 1.13 * eg + 8 * U * (1 + np.abs(a))), (da, 0.8 * eg + 8 * U * (1 + np.abs(g))), (u, eu)


def gated(x, wg, wu, act, kind):
    (a, ea), _, (u, eu) = _projections(x, wg, wu, act)
    return _rounded(a * u, ea * np.abs(u) + np.abs(a) * eu + ea * eu + 2 * U * np.abs(a * u), kind)


def gated_backward(x, wg, wu, dout, act, kind):
    """{"dx", "dw_gate", "dw_up"}; dg and du enter their products rounded to the
    rows' type."""
    n, H = x.shape[0], wg.shape[0]
    (a, ea), (da, eda), (u, eu) = _projections(x, wg, wu, act)
    ro = UB if kind == "bf16" else 0.0
    dg, du = dout * u * da, dout * a
    edg = np.abs(dout) * (eu * np.abs(da) + np.abs(u) * eda + eu * eda) + 3 * U * np.abs(dg)
    edu = np.abs(dout) * ea + 2 * U * np.abs(du)
    edg, edu = edg + ro * (np.abs(dg) + edg), edu + ro * (np.abs(du) + edu)
    dx = dg @ wg + du @ wu
    edx = edg @ np.abs(wg) + edu @ np.abs(wu) + (2 * H + 2) * U * ((np.abs(dg) + edg) @ np.abs(wg) + (np.abs(du) + edu) @ np.abs(wu))
    got = {"dx": _rounded(dx, edx, kind)}
    for name, d, ed in (("dw_gate", dg, edg), ("dw_up", du, edu)):
        e = ed.T @ np.abs(x) + (n + 2) * U * ((np.abs(d) + ed).T @ np.abs(x))
        got[name] = _rounded(d.T @ x, e, kind)
    return got
