"""Plain implementations for the tests of the rotary positions, the paged cache
and its attention: numpy on the host, written from include/w4.h.

The record layout is restated value by value (`key_at`, `value_at`), the
quantiser in fp32 with every operation rounded once (so its codes are the
library's bit for bit), the rotation in fp32 likewise, and the attention in
fp64 over the values that the cache holds.

Tolerances of the attention (`check_attention`), with A = sum_j p_j |v_j| (fp64):
  * probabilities enter the second product rounded to bfloat16 (relative error
    at most 2^-8) or binary16 scaled into its range (2^-11, and for
    probabilities under 2^-20 of the largest the subnormal spacing: in all at
    most 2^-10): u_p * A;
  * a score's fp32 sum has an error of at most dS = (D + 4) 2^-23 scale M,
    M the sum of the magnitudes that are added (|q k| for bf16; for the codes
    s (1024 + 2 * 255) |q|, the codes' fp16 form); exp turns it into a relative
    error of 2 dS of every p and of their sum: 4 dS A;
  * fp32 sums of n terms, exponentials within 2^-21, the joins: (n + 64) 2^-23 A;
  * a bfloat16 result rounds by at most 2^-8 of itself.
The dS term is a worst case; rounding errors of both signs stay far below it,
so the 2-norm of all errors must also be within (u_p + 2^-8 [bf16] + 2^-12) times
the 2-norm of A.
"""
from __future__ import annotations

import numpy as np

FMT = {"bf16": 0, "int8": 1, "int4": 2}
LEVELS = {"int8": 255, "int4": 15}


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """fp32 -> bfloat16 bit patterns, nearest even (NaN stays NaN)."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((b.astype(np.uint64) + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32)


def bf16(x: np.ndarray) -> np.ndarray:
    return bf16_value(bf16_bits(x))


def record_bytes(fmt: str, D: int) -> int:
    return {"bf16": 64 * D, "int8": 32 * D + 128, "int4": 16 * D + 128}[fmt]


def key_at(fmt: str, D: int, r: int, d: int):
    """(byte, nibble) of value d of token r's key in its record."""
    if fmt == "bf16":
        return r * 2 * D + ((d // 8) ^ (r & 7)) * 16 + d % 8 * 2, 0
    if fmt == "int8":
        piece = d // 16
        if D == 128:
            piece ^= 4 * (r & 1)
        return r * D + piece * 16 + d % 16, 0
    return r * (D // 2) + d // 2, d & 1


def value_at(fmt: str, D: int, r: int, d: int):
    if fmt == "bf16":
        return 32 * D + key_at(fmt, D, r, d)[0], 0
    lane, byte = 4 * (d & 7) + (r & 7) // 2, 2 * (r & 1) + r // 8
    if fmt == "int8":
        return 16 * D + d // 32 * 512 + lane * 16 + d // 8 % 4 * 4 + byte, 0
    return 8 * D + d // 64 * 512 + lane * 16 + d // 16 % 4 * 4 + byte, d // 8 & 1


_PLACES = {}


def places(fmt: str, D: int):
    """Byte and nibble of every (token, value): keys, then values."""
    if (fmt, D) not in _PLACES:
        _PLACES[fmt, D] = [np.array([[f(fmt, D, r, d) for d in range(D)] for r in range(16)])
                           for f in (key_at, value_at)]
    return _PLACES[fmt, D]


def quantise(x: np.ndarray, fmt: str):
    """(codes uint8 [.., D], scale binary16 [..], zero [..]) of fp32 rows."""
    top = np.float32(LEVELS[fmt])
    lo = np.minimum(x.min(-1), np.float32(0))
    hi = np.maximum(x.max(-1), np.float32(0))
    s16 = np.minimum((hi - lo) * (np.float32(1) / top), np.float32(65504)).astype(np.float16)
    s = s16.astype(np.float32)
    safe = np.where(s == 0, np.float32(1), s)
    z = np.where(s == 0, np.float32(0), np.clip(np.rint(-lo / safe), 0, top))
    q = np.clip(np.rint(x / safe[..., None]) + z[..., None], 0, top)
    q = np.where(s[..., None] == 0, 0, q)
    return q.astype(np.uint8), s16, z.astype(np.uint16)


def held(x: np.ndarray, fmt: str) -> np.ndarray:
    """The fp32 values that a cache of this format holds for rows x."""
    if fmt == "bf16":
        return bf16(x)
    q, s, z = quantise(x, fmt)
    return (q.astype(np.float32) - z[..., None].astype(np.float32)) * \
        s[..., None].astype(np.float32)


class Pool:
    """A pool in host memory, byte for byte; starts as `fill` everywhere."""

    def __init__(self, fmt, D, kv_heads, page_tokens, pages, fill=0xFF):
        self.fmt, self.D, self.H, self.P, self.pages = fmt, D, kv_heads, page_tokens, pages
        self.nb = record_bytes(fmt, D)
        self.bytes = np.full((pages, kv_heads, page_tokens // 16, self.nb), fill, np.uint8)

    def _rec(self, page, in_page):
        return self.bytes[page, :, in_page // 16], in_page % 16

    def write(self, page, in_page, k, v):
        """k, v: fp32 [kv_heads, D] of one token."""
        rec, r = self._rec(page, in_page)
        for which, x in enumerate((k, v)):
            at = places(self.fmt, self.D)[which][r]
            if self.fmt == "bf16":
                bits = bf16_bits(x)
                rec[:, at[:, 0]] = (bits & 255).astype(np.uint8)
                rec[:, at[:, 0] + 1] = (bits >> 8).astype(np.uint8)
                continue
            q, s, z = quantise(x, self.fmt)
            if self.fmt == "int8":
                rec[:, at[:, 0]] = q
            else:
                for n in (0, 1):
                    m = at[:, 1] == n
                    b = at[m, 0]
                    rec[:, b] = (rec[:, b] & (0xF0 if n == 0 else 0x0F)) | (q[:, m] << (4 * n))
            o = self.nb - 128 + 64 * which + 4 * r
            rec[:, o:o + 2] = s.view(np.uint16)[:, None].view(np.uint8).reshape(self.H, 2)
            rec[:, o + 2:o + 4] = z[:, None].view(np.uint8).reshape(self.H, 2)

    def read(self, page, in_page):
        """fp32 (k, v) [kv_heads, D] of one token."""
        rec, r = self._rec(page, in_page)
        out = []
        for which in (0, 1):
            at = places(self.fmt, self.D)[which][r]
            if self.fmt == "bf16":
                bits = rec[:, at[:, 0]].astype(np.uint16) | \
                    (rec[:, at[:, 0] + 1].astype(np.uint16) << 8)
                out.append(bf16_value(bits))
                continue
            q = rec[:, at[:, 0]]
            if self.fmt == "int4":
                q = (q >> (4 * at[:, 1]).astype(np.uint8)) & 15
            o = self.nb - 128 + 64 * which + 4 * r
            m = np.ascontiguousarray(rec[:, o:o + 4])
            s = m[:, :2].copy().view(np.float16).astype(np.float32)
            z = m[:, 2:].copy().view(np.uint16).astype(np.float32)
            out.append((q.astype(np.float32) - z) * s)
        return out


def rotate(x, positions, table, layout):
    """fp32 rotation with every operation rounded once; table fp32 [rows, n, 2]."""
    x = np.asarray(x, np.float32)
    n = table.shape[1]
    cs = table[np.abs(positions)][:, None]
    c, s = cs[..., 0], cs[..., 1] * np.where(positions < 0, -1, 1).astype(np.float32)[:, None, None]
    y = x.copy()
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == 0 else (slice(0, 2 * n, 2),
                                                               slice(1, 2 * n, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def attention(q, keys, values, lens, tokens, scale, window):
    """fp64 attention.  q fp32 [seqs * tokens, q_heads, D]; keys, values: per
    sequence fp32 [len, kv_heads, D].  Returns out, lse, A = sum_j p_j |v_j|."""
    T, H, D = q.shape
    out, mag = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        k, v = keys[b].astype(np.float64), values[b].astype(np.float64)
        R = H // k.shape[1]
        for i in range(tokens):
            last = n - tokens + i
            first = max(0, last - window + 1) if window else 0
            if last < first:
                continue
            for h in range(H):
                x = k[first:last + 1, h // R] @ q[b * tokens + i, h].astype(np.float64) * scale
                m = x.max()
                e = np.exp(x - m)
                total = e.sum()
                t = b * tokens + i
                out[t, h] = e @ v[first:last + 1, h // R] / total
                mag[t, h] = e @ np.abs(v[first:last + 1, h // R]) / total
                lse[t, h] = m + np.log(total)
    return out, lse, mag


def score_error(fmt, q, keys, scales, lens, scale):
    """dS of the module's note: a bound on any score's fp32 error."""
    D, worst = q.shape[2], 0.0
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        if fmt == "bf16":
            m = np.abs(q).max() * np.abs(keys[b]).sum(-1).max()
        else:
            m = scales[b].max() * (1024 + 510) * np.abs(q).sum(-1).max()
        worst = max(worst, float(m))
    return (D + 4) * 2.0 ** -23 * abs(scale) * worst


def check_attention(got, lse, ref, ref_lse, mag, fmt, dS, n, bf16_out, what=""):
    u_p = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -10
    out = 2.0 ** -8 if bf16_out else 0.0
    err = np.abs(got.astype(np.float64) - ref)
    bound = (u_p + 4 * dS + (n + 64) * 2.0 ** -23) * mag + out * np.abs(ref) + 1e-30
    assert np.isfinite(got).all(), what
    assert (err <= bound).all(), (what, float((err / bound).max()))
    size = np.linalg.norm(mag)
    if size:
        assert np.linalg.norm(err) <= (u_p + out + 2.0 ** -12) * size, \
            (what, float(np.linalg.norm(err) / size))
    seen = np.isfinite(ref_lse)
    assert (np.isneginf(lse) == ~seen).all(), what
    # lse: the scores' error, and the fp32 sum and logarithm
    lim = 2 * dS + (n + 64) * 2.0 ** -23 + 2.0 ** -22 * np.abs(ref_lse[seen])
    assert (np.abs(lse[seen] - ref_lse[seen]) <= lim).all(), \
        (what, float((np.abs(lse[seen] - ref_lse[seen]) / lim).max()))
