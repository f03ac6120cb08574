"""The attention's close bounds, on the host: exact results and an fp32
evaluation pass, small mistakes do not, those in the log-sum-exp alone among
them."""
import numpy as np
import pytest

from tests import attn_bounds as ab
from tests import kv_testutil as kv

N, M, H, R = 500, 2, 2, 4


def problem(fmt, D, window=0):
    rng = np.random.default_rng(D)
    chan = np.where(rng.random((H, D)) < 1 / 16, 4, 1).astype(np.float32)
    k0 = kv.bf16(rng.standard_normal((N, H, D)).astype(np.float32) * chan)
    v0 = kv.bf16(rng.standard_normal((N, H, D)).astype(np.float32) + 0.25)
    q = kv.bf16(rng.standard_normal((M, H * R, D)).astype(np.float32))
    codes = None if fmt == "bf16" else [tuple(np.asarray(x, np.float64)
                                              for x in kv.quantise(k0, fmt))]
    return dict(q=q, keys=[kv.held(k0, fmt)], values=[kv.held(v0, fmt)], lens=[N], tokens=M,
                scale=D ** -0.5, window=window), codes


def fp32(fmt, a, codes, added=0):
    """The kernel's arithmetic in fp32, 16 products at a time; added: a number
    that stays in the codes (as their 16-bit form would have it)."""
    f = np.float32
    q, T = a["q"], a["q"].shape[0]
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for t, h in np.ndindex(T, H * R):
        n = N - M + t + 1
        v, qq = a["values"][0][:n, h // R], q[t, h]
        if fmt == "bf16":
            u, s, z = a["keys"][0][:n, h // R], np.ones(n, f), np.zeros(n, f)
        else:
            u, s, z = (x[:n, h // R].astype(f) for x in codes[0])
        total = f(0)
        for d in range(len(qq)):
            total = f(total + qq[d])
        acc = f(-1) * (z if not added else f(0)) * total
        for d in range(0, len(qq), 16):
            part = (u[:, d:d + 16].astype(np.float64) + added) @ qq[d:d + 16].astype(np.float64)
            acc = (acc + part).astype(f)
        if added:
            acc = (acc - (f(added) + z) * total).astype(f)
        x = (acc * s * f(a["scale"])).astype(f)
        e = np.exp(x - x.max()).astype(f)
        lse[t, h] = x.max() + np.log(e.sum(dtype=np.float64))
        p = e.astype(np.float16).astype(f) if fmt != "bf16" else e
        out[t, h] = p @ v / e.sum()
    return out, lse


def wrong(a, codes, fmt, mistake):
    b = dict(a)
    out, lse, _ = kv.attention(**a)
    if mistake == "lse of every row":
        lse = lse + 5e-4
    elif mistake == "lse of one row":
        lse[1, 3] -= 5e-3
    elif mistake == "lse without one key":
        lse = kv.attention(**{**a, "window": N - M})[1]
    elif mistake == "window":
        out, lse, _ = kv.attention(**{**a, "window": N - M})
    elif mistake == "scale":
        out, lse, _ = kv.attention(**{**a, "scale": a["scale"] * 1.002})
    elif mistake == "a value":
        b["values"] = [a["values"][0].copy()]
        b["values"][0][17] *= 2
        out, _, _ = kv.attention(**b)
    elif mistake == "a head's keys":
        b["keys"] = [a["keys"][0][:, ::-1]]
        out, lse, _ = kv.attention(**b)
    return out, lse


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D", [64, 128])
def test_exact_and_fp32_results_pass(fmt, D):
    a, codes = problem(fmt, D)
    rows = ab.rows_of(fmt, codes=codes, **a)
    out, lse, _ = kv.attention(**a)
    ab.check(out, lse, rows, fmt, False)
    out, lse = fp32(fmt, a, codes)
    ab.check(out, lse, rows, fmt, False)
    ab.check(kv.bf16(out.astype(np.float32)), lse, rows, fmt, True)


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mistake", ["lse of every row", "lse of one row", "lse without one key",
                                     "window", "scale", "a value", "a head's keys"])
def test_planted_mistakes_leave_the_bound(fmt, D, mistake):
    a, codes = problem(fmt, D)
    rows = ab.rows_of(fmt, codes=codes, **a)
    out, lse = wrong(a, codes, fmt, mistake)
    with pytest.raises(AssertionError):
        ab.check(out, lse, rows, fmt, False)


@pytest.mark.parametrize("D", [64, 128])
def test_coarse_probabilities_beside_bf16_values_leave_the_bound(D):
    a, _ = problem("bf16", D)
    rows = ab.rows_of("bf16", codes=None, **a)
    out, lse, _ = kv.attention(**a)
    for t, h in np.ndindex(*lse.shape):
        n = N - M + t + 1
        p = np.exp(a["keys"][0][:n, h // R] @ a["q"][t, h].astype(np.float64) * a["scale"]
                   - lse[t, h]).astype(np.float32)
        out[t, h] = kv.bf16(p).astype(np.float64) @ a["values"][0][:n, h // R]
    with pytest.raises(AssertionError):
        ab.check(out, lse, rows, "bf16", False)


def test_rows_that_see_nothing():
    a, codes = problem("int4", 64)
    a["lens"], a["keys"], a["values"] = [1], [a["keys"][0][:1]], [a["values"][0][:1]]
    rows = ab.rows_of("int4", codes=[tuple(x[:1] for x in codes[0])], **a)
    out, lse, _ = kv.attention(**a)
    ab.check(out, lse, rows, "int4", False)
    out[0, 0, 0] = 1e-3
    with pytest.raises(AssertionError):
        ab.check(out, lse, rows, "int4", False)
