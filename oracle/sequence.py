"""Oracle of the attention over behaviour sequences (test infrastructure only:
imported by the tests, never by the library or its binding).

Plain numpy in float64, one sequence, head and formula at a time, with no
running maximum, no tiles and no cache pages.  Next to each result stands a
bound of how far an implementation in fp32 (or with bf16 products) may be from
it, from the standard model of rounded arithmetic: a sum of n products is off
by at most n u times the sum of their magnitudes, u = 2^-24.
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24          # unit roundoff of fp32
UB = 2.0 ** -8          # unit roundoff of bf16: 8 significant bits, to nearest
# rounding of a factor before a product; "bf16 pairs": the factor as the sum of
# two bf16 values, the second one the rounded remainder of the first
R = {"f32": 0.0, "bf16": UB, "bf16 pairs": UB * UB}
TERMS = {"f32": 1, "bf16": 1, "bf16 pairs": 2}
OUT = {"f32": U, "bf16": UB, "bf16 pairs": UB}


def bucket(pos_i, pos_j, boundaries):
    """Number of boundaries <= the distance saturated to int32, one by one."""
    d = np.clip(np.asarray(pos_i, np.int64) - np.asarray(pos_j, np.int64), -2**31, 2**31 - 1)
    b = np.zeros(d.shape, np.int64)
    for m in boundaries:
        b += (m <= d)
    return b


def _one(q, k, v, pos, bias, key_off, boundaries, causal, scale, do=None):
    """One sequence and head: every matrix of the formulas, and bounds."""
    n, D = q.shape
    cell = bucket(pos[:, None], pos[None, :], boundaries)
    see = np.ones((n, n), bool)
    if causal:
        see &= np.tril(see)
    if key_off is not None:
        see &= (key_off >= 0)[None, :]
    k = np.where(see.any(0)[:, None], k, 0.0)    # what nobody sees is not used
    v = np.where(see.any(0)[:, None], v, 0.0)
    see &= bias[cell] > -1e30                    # a bias that hides its pairs; their k and v are still read
    bias = np.where(bias > -1e30, bias, 0.0)
    s = scale * (q @ k.T) + bias[cell]
    # an exponent's error: D products, the scale, the bias, the difference
    # from the row's statistic, the conversion to base 2
    es = U * ((D + 4) * abs(scale) * (np.abs(q) @ np.abs(k).T) + 4 * np.abs(s) + 4 * np.abs(bias[cell]) + 8)
    s = np.where(see, s, -np.inf)
    top = s.max(1, initial=-np.inf)
    p = np.where(see, np.exp(s - np.where(np.isinf(top), 0.0, top)[:, None]), 0.0)
    total = p.sum(1)
    p = p / np.where(total == 0, 1.0, total)[:, None]
    lse = np.where(total == 0, -np.inf, top + np.log(np.where(total == 0, 1.0, total)))
    worst = np.where(see, es, 0.0).max(1, initial=0.0)
    ep = 2 * worst + (2 * n + 16 + 4 * np.abs(np.where(np.isinf(lse), 0.0, lse))) * U      # relative, every p of a row
    got = {"cell": cell, "see": see, "p": p, "lse": lse, "ep": ep, "k": k, "v": v}
    if do is not None:
        dp = do @ v.T
        edp = (D + 2) * U * (np.abs(do) @ np.abs(v).T)
        delta = (p * dp).sum(1)
        edelta = (p * (ep[:, None] * np.abs(dp) + edp)).sum(1) + (n + 2) * U * (p * np.abs(dp)).sum(1)
        # the same sum as dout . out: the rounding of out enters
        ds = p * (dp - delta[:, None])
        got |= {"ds": ds, "eds": ep[:, None] * np.abs(ds) + p * (edp + edelta[:, None] + 2 * U * np.abs(dp))}
    return got


def attention(q, k, v, pos, bias, offsets, boundaries, causal, scale, key_off=None, dout=None, kind="f32"):
    """q [N, H, D], k, v [N, Hk, D], bias [H, nb] (any float type holding the
    exact inputs).  Returns a dict name -> (value, bound)."""
    q, k, v, bias = (np.asarray(x, np.float64) for x in (q, k, v, bias))
    N, H, D = q.shape
    Hk = k.shape[1]
    r, ro, terms = R[kind], OUT[kind], TERMS[kind]
    zeros = lambda *s: [np.zeros(s), np.zeros(s)]  # noqa: E731
    out = zeros(N, H, D)
    lse = np.full((H, N), -np.inf)
    dq, dk, dv, db = zeros(N, H, D), zeros(N, Hk, D), zeros(N, Hk, D), zeros(H, bias.shape[1])
    if dout is not None:
        dout = np.asarray(dout, np.float64)
    for a, e in zip(offsets[:-1], offsets[1:]):
        a, e, n = int(a), int(e), int(e - a)
        if n == 0:
            continue
        for h in range(H):
            g = h // (H // Hk)
            ko = None if key_off is None else key_off[a:e]
            m = _one(q[a:e, h], k[a:e, g], v[a:e, g], pos[a:e], bias[h], ko, boundaries, causal, scale,
                     None if dout is None else dout[a:e, h])
            p, ep = m["p"], m["ep"][:, None]
            out[0][a:e, h] = p @ m["v"]
            out[1][a:e, h] = (ep + terms * n * U + r) * (p @ np.abs(m["v"]))
            lse[h, a:e] = m["lse"]
            if dout is None:
                continue
            do, ds, eds = dout[a:e, h], m["ds"], m["eds"]
            sums = (terms * len(q) * (H // Hk) + 4) * U       # at most that many terms in a key's sums
            dq[0][a:e, h] = scale * (ds @ m["k"])
            dq[1][a:e, h] = abs(scale) * ((eds + (r + (terms * n + 2) * U) * np.abs(ds)) @ np.abs(m["k"]))
            dk[0][a:e, g] += scale * (ds.T @ q[a:e, h])
            dk[1][a:e, g] += abs(scale) * ((eds + (r + sums) * np.abs(ds)).T @ np.abs(q[a:e, h]))
            dv[0][a:e, g] += p.T @ do
            dv[1][a:e, g] += (p * (ep + r + sums)).T @ np.abs(do)
            np.add.at(db[0][h], m["cell"][m["see"]], ds[m["see"]])
            count = np.bincount(m["cell"][m["see"]], minlength=bias.shape[1])
            np.add.at(db[1][h], m["cell"][m["see"]], (eds + count[m["cell"]] * U * np.abs(ds))[m["see"]])
    tiny = 1e-30
    got = {"out": (out[0], out[1] + ro * np.abs(out[0]) + tiny), "lse": lse}
    if dout is not None:
        got |= {"dq": (dq[0], dq[1] + ro * np.abs(dq[0]) + tiny), "dk": (dk[0], dk[1] + ro * np.abs(dk[0]) + tiny),
                "dv": (dv[0], dv[1] + ro * np.abs(dv[0]) + tiny), "dbias": (db[0], db[1] + 2 * U * np.abs(db[0]) + tiny)}
    return got


def step(histories, q, bias, boundaries, scale, kind="f32"):
    """histories: per user (k [n, Hk, D], v, pos [n]) with the new event last,
    or None for an idle one.  Returns (out [B, H, D], bound)."""
    B, H, D = q.shape
    out, err = np.zeros((B, H, D)), np.zeros((B, H, D))
    for b, hist in enumerate(histories):
        if hist is None:
            continue
        k, v, pos = (np.asarray(x, np.float64) if x.ndim > 1 else np.asarray(x) for x in hist)
        n, group = len(k), H // k.shape[1]
        for h in range(H):
            row = np.zeros((n, D))
            row[-1] = q[b, h]
            m = _one(row, k[:, h // group], v[:, h // group], pos, np.asarray(bias[h], np.float64), None, boundaries,
                     False, scale)
            p = m["p"][-1]
            out[b, h] = p @ m["v"]
            err[b, h] = (m["ep"][-1] + TERMS[kind] * n * U + R[kind]) * (p @ np.abs(m["v"])) + OUT[kind] * np.abs(out[b, h]) + 1e-30
    return out, err


def assign(counts, lens, table, free, page_size):
    """(slots, offsets, pages taken, table) in Python integers."""
    table = [list(map(int, row)) for row in table]
    slots, offsets, taken = [], [0], 0
    for b, (c, n) in enumerate(zip(counts, lens)):
        for e in range(int(n), int(n) + int(c)):
            if e % page_size == 0:               # the first event of a page takes the next free one
                table[b][e // page_size] = int(free[taken])
                taken += 1
            slots.append(table[b][e // page_size] * page_size + e % page_size)
        offsets.append(len(slots))
    return slots, offsets, taken, table
