"""Bounds of the paged attention's errors from the magnitudes that the kernel
adds up, close enough to tell a wrong log-sum-exp apart (kv_testutil's bound
takes codes with 1024 added to them, which the kernel's keys do not have: for
quantised caches it lets a log-sum-exp pass that is off by 0.05 to 0.8).

A score is a sum of D products and a start, in fp32, in an order and with a
rounding that are the tensor cores' own ("at least single precision": a
relative 2^-23 of the partial sum for each addition):
  * bf16:  sum q_d k_d;  codes: s (sum q_d u_d - z sum q), the second sum a
    start value with up to D roundings of its own.
  * The partial sums of terms of both signs stay within three times their
    2-norm of a line from the start to the end: within
      R = |sum q k| + 3 |q k|_2                              (bf16)
      R = s (|z sum q| + |sum q u| + 3 |q u|_2 + 3 z |q|_2)  (codes)
    so a score is within dS = |scale| 2^-23 D R of the exact one if all D
    errors have one sign, and within dS / sqrt(D) as a root mean square if
    they have both, or only the D / 16 additions between products do err (those
    inside one are exact there).
  * A further 4 roundings of the score itself: 2^-21 |score|.
Log-sum-exp: sum_j p_j dS_j; the approximate exponential and logarithms (2^-22
each, the logarithm of a value's scale up to 24 in size); sums over n keys, of
which a lane adds every eighth, then the warps and pieces.
Result: a change of the scores by dS changes it by at most 2 max dS (A + |o|),
A = sum_j p_j |v_j|; probabilities are rounded by at most u_p of themselves, of
both signs, so in the 2-norm by u_p sqrt(sum_j p_j^2 v_j^2).
"""
from __future__ import annotations

import numpy as np

from tests import kv_testutil as kv

U_P = {"bf16": 2.0 ** -15, "int8": 2.0 ** -10, "int4": 2.0 ** -10}


class Row:
    """What the bounds of one row (new token and head) need."""

    def __init__(self, fmt, q, k, v, codes, scale):
        """q [D]; k, v fp64 [n, D]; codes: (u [n, D], s [n], z [n]) or None."""
        D = len(q)
        x = k @ q * scale
        top = x.max()
        e = np.exp(x - top)
        p = e / e.sum()
        self.lse, self.out = top + np.log(e.sum()), p @ v
        self.mag, self.rms_p = p @ np.abs(v), np.sqrt(np.square(p) @ np.square(v))
        if fmt == "bf16":
            R = np.abs(k @ q) + 3 * np.sqrt(np.square(k) @ np.square(q))
        else:
            u, s, z = codes
            R = s * (np.abs(z * q.sum()) + np.abs(u @ q)
                     + 3 * np.sqrt(np.square(u) @ np.square(q)) + 3 * z * np.linalg.norm(q))
        dS = abs(scale) * 2.0 ** -23 * D * R
        self.mean_dS = float(p @ dS) + 2.0 ** -21 * abs(float(p @ np.abs(x)))
        self.max_dS = float((dS + 2.0 ** -21 * np.abs(x)).max())
        self.rms_dS = float(p @ dS) / D ** 0.5 + 2.0 ** -21 * float(p @ np.abs(x))
        self.n = len(k)


def rows_of(fmt, q, keys, values, codes, lens, tokens, scale, window):
    """Row or None (sees nothing) of every [token, head].  Arguments as for
    kv.attention; codes: per sequence (u [n, kv_heads, D], s, z [n, kv_heads])."""
    T, H, _ = q.shape
    rows = np.full((T, H), None, object)
    for b, n in enumerate(lens):
        R = H // keys[b].shape[1]
        for i in range(tokens):
            last = n - tokens + i
            first = max(0, last - window + 1) if window else 0
            if n <= 0 or last < first:
                continue
            at = slice(first, last + 1)
            for h in range(H):
                c = codes and tuple(y[at, h // R].astype(np.float64) for y in codes[b])
                rows[b * tokens + i, h] = Row(
                    fmt, q[b * tokens + i, h].astype(np.float64),
                    keys[b][at, h // R].astype(np.float64),
                    values[b][at, h // R].astype(np.float64), c, scale)
    return rows


def check(got, lse, rows, fmt, bf16_out, what=""):
    """got [T, H, D], lse [T, H] against the rows' exact values."""
    u_p, rounding = U_P[fmt], 2.0 ** -8 if bf16_out else 0.0
    err2 = lim2 = lse2 = lse_lim2 = 0.0
    count = 0
    for t, h in np.ndindex(rows.shape):
        r = rows[t, h]
        if r is None:
            assert (got[t, h] == 0).all() and np.isneginf(lse[t, h]), what
            continue
        sums = (r.n / 8 + 64) * 2.0 ** -23
        off = abs(float(lse[t, h]) - r.lse)
        assert off <= r.mean_dS + sums + 2.0 ** -22 * (abs(r.lse) + 24), (what, t, h, off)
        err = np.abs(got[t, h].astype(np.float64) - r.out)
        size = r.mag + np.abs(r.out)
        assert (err <= u_p * r.mag + (2 * r.max_dS + sums + 2.0 ** -20) * size
                + rounding * np.abs(r.out) + 1e-30).all(), (what, t, h, (err / size).max())
        lse2 += off ** 2
        lse_lim2 += (r.rms_dS + 2.0 ** -20 + 2.0 ** -23 * abs(r.lse)) ** 2
        err2 += np.square(err).sum()
        lim2 += np.square(2 * u_p * r.rms_p + (2 * r.rms_dS + 2.0 ** -20) * size
                          + rounding * np.abs(r.out)).sum()
        count += 1
    assert lse2 <= lse_lim2, (what, "lse", (lse2 / max(count, 1)) ** 0.5,
                              (lse_lim2 / max(count, 1)) ** 0.5)
    assert err2 <= lim2, (what, "out", (err2 / lim2) ** 0.5)


def pool_codes(host, table, n):
    """(u, s, z) of tokens 0 .. n - 1 whose pages a row of the table gives."""
    D, H = host.D, host.H
    u, s, z = np.zeros((n, H, D)), np.zeros((n, H)), np.zeros((n, H))
    for t in range(n):
        rec, r = host._rec(table[t // host.P], t % host.P)
        at = kv.places(host.fmt, D)[0][r]
        c = rec[:, at[:, 0]]
        u[t] = (c >> (4 * at[:, 1]).astype(np.uint8)) & 15 if host.fmt == "int4" else c
        m = np.ascontiguousarray(rec[:, host.nb - 128 + 4 * r:host.nb - 124 + 4 * r])
        s[t] = m[:, :2].copy().view(np.float16)[:, 0]
        z[t] = m[:, 2:].copy().view(np.uint16)[:, 0]
    return u, s, z
