"""Host-side checks of the rotary, paged-cache and attention calls that need no
GPU: sizes, argument errors (every call here fails validation, so no pointer is
looked at), and the tests' own plain implementations."""
import ctypes

import numpy as np
import pytest

from tests import kv_testutil as kv
from tests.test_abi_host import FAKE, lib  # noqa: F401

P, I, I64, D64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double


class Heads(ctypes.Structure):
    _fields_ = [("data", P), ("token_stride", I64), ("head_stride", I64)]


class Rotation(ctypes.Structure):
    _fields_ = [("table", P), ("rows", I), ("rotary_dim", I), ("layout", I)]


class Spec(ctypes.Structure):
    _fields_ = [("rotary_dim", I), ("scaling", I), ("base", D64), ("factor", D64),
                ("original_context", D64), ("low_turns", D64), ("high_turns", D64),
                ("amplitude", D64)]


class Cache(ctypes.Structure):
    _fields_ = [("pool", P), ("format", I), ("kv_heads", I), ("head_dim", I),
                ("page_tokens", I), ("pages", I), ("error", P)]


class Table(ctypes.Structure):
    _fields_ = [("pages", P), ("seqs", I), ("width", I), ("stride", I64)]


def ref(s):
    return None if s is None else ctypes.byref(s)


def cache(**kw):
    a = dict(pool=FAKE, format=2, kv_heads=2, head_dim=64, page_tokens=16, pages=4, error=None)
    a.update(kw)
    return Cache(*a.values())


def heads(data=FAKE, token=128, head=64):
    return Heads(data, token, head)


def table(pages=FAKE, seqs=1, width=4, stride=4):
    return Table(pages, seqs, width, stride)


@pytest.mark.parametrize("fmt,D,want", [(0, 128, 8192), (0, 64, 4096), (1, 128, 4224),
                                        (1, 64, 2176), (2, 128, 2176), (2, 64, 1152)])
def test_pool_bytes(lib, fmt, D, want):  # noqa: F811
    n = ctypes.c_size_t()
    c = cache(format=fmt, head_dim=D, kv_heads=3, page_tokens=48, pages=70000)
    assert lib.w4_kv_pool_bytes(ref(c), ctypes.byref(n)) == 0
    assert n.value == 70000 * 3 * 3 * want
    assert kv.record_bytes({v: k for k, v in kv.FMT.items()}[fmt], D) == want


@pytest.mark.parametrize("kw,want", [
    (dict(format=3), 1), (dict(format=-1), 1), (dict(kv_heads=0), 1), (dict(pages=0), 1),
    (dict(page_tokens=0), 1), (dict(page_tokens=8), 1), (dict(page_tokens=24), 1),
    (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(head_dim=256), 2)])
def test_cache_errors(lib, kw, want):  # noqa: F811
    n = ctypes.c_size_t()
    assert lib.w4_kv_pool_bytes(ref(cache(**kw)), ctypes.byref(n)) == want
    assert append(lib, c=cache(**kw)) == want
    assert read(lib, c=cache(**kw)) == want
    assert attn(lib, c=cache(**kw)) == want
    assert lib.w4_kv_pool_bytes(None, ctypes.byref(n)) == 1
    assert lib.w4_kv_pool_bytes(ref(cache()), None) == 1


def spec(**kw):
    a = dict(rotary_dim=64, scaling=0, base=1e4, factor=1.0, original_context=0.0, low_turns=0.0,
             high_turns=0.0, amplitude=1.0)
    a.update(kw)
    return Spec(*a.values())


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=514), dict(scaling=4),
    dict(scaling=-1), dict(base=0.0), dict(base=float("nan")), dict(base=float("inf")),
    dict(scaling=1, factor=0.0), dict(scaling=1, factor=float("inf")),
    dict(amplitude=float("nan")), dict(scaling=3, factor=2.0),
    dict(scaling=3, factor=2.0, original_context=4096.0, low_turns=2.0, high_turns=2.0)])
def test_rope_table_errors(lib, kw):  # noqa: F811
    lib.w4_rope_table.argtypes = [P, I, P, P]
    assert lib.w4_rope_table(ref(spec(**kw)), 10, FAKE, None) == 1
    assert lib.w4_rope_table(None, 10, FAKE, None) == 1
    assert lib.w4_rope_table(ref(spec()), 0, FAKE, None) == 1
    assert lib.w4_rope_table(ref(spec()), 10, None, None) == 1
    assert lib.w4_rope_table(ref(spec()), 10, FAKE + 4, None) == 1


def rope(lib, x=heads(), y=heads(), tokens=1, nheads=2, D=64, pos=FAKE,  # noqa: F811
         rot=Rotation(FAKE, 10, 64, 0), error=None):
    lib.w4_rope.argtypes = [P, P, I, I, I, P, P, P, P]
    return lib.w4_rope(ref(x), ref(y), tokens, nheads, D, pos, ref(rot), error, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(rot=None), 1), (dict(tokens=-1), 1),
    (dict(nheads=0), 1), (dict(D=0), 1), (dict(D=1025), 1), (dict(D=62), 1), (dict(pos=None), 1),
    (dict(pos=FAKE + 2), 1), (dict(error=FAKE + 2), 1), (dict(x=heads(None)), 1),
    (dict(y=heads(FAKE + 1)), 1), (dict(rot=Rotation(None, 10, 64, 0)), 1),
    (dict(rot=Rotation(FAKE + 8, 10, 64, 0)), 1), (dict(rot=Rotation(FAKE, 0, 64, 0)), 1),
    (dict(rot=Rotation(FAKE, 10, 63, 0)), 1), (dict(rot=Rotation(FAKE, 10, 64, 2)), 1),
    (dict(tokens=1 << 30, nheads=2), 2), (dict(tokens=0, pos=None), 0)])
def test_rope_errors(lib, kw, want):  # noqa: F811
    assert rope(lib, **kw) == want


def append(lib, c=cache(), k=heads(), v=heads(), q=None, qo=None, hq=0, tokens=1,  # noqa: F811
           pos=FAKE, seq=None, t=table(), rot=None):
    lib.w4_kv_append.argtypes = [P, P, P, P, P, I, I, P, P, P, P, P]
    return lib.w4_kv_append(ref(c), ref(k), ref(v), ref(q), ref(qo), hq, tokens, pos, seq, ref(t),
                            ref(rot), None)


ROT = Rotation(FAKE, 10, 64, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(c=None), 1), (dict(c=cache(pool=None)), 1), (dict(c=cache(pool=FAKE + 64)), 1),
    (dict(c=cache(error=FAKE + 1)), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(k=heads(None)), 1), (dict(v=heads(FAKE + 8)), 1), (dict(k=heads(token=129)), 1),
    (dict(k=heads(head=60)), 1), (dict(tokens=-1), 1), (dict(pos=None), 1),
    (dict(pos=FAKE + 1), 1), (dict(seq=FAKE + 2), 1), (dict(t=None), 1),
    (dict(t=table(None)), 1), (dict(t=table(seqs=0)), 1), (dict(t=table(width=0)), 1),
    (dict(t=table(stride=3)), 1), (dict(t=table(seqs=2)), 1), (dict(q=heads()), 1),
    (dict(qo=heads()), 1), (dict(q=heads(), qo=heads(), hq=0, rot=ROT), 1),
    (dict(q=heads(None), qo=heads(), hq=2, rot=ROT), 1),
    (dict(q=heads(), qo=heads(FAKE + 2), hq=2, rot=ROT), 1),
    (dict(rot=Rotation(FAKE, 10, 24, 0)), 1), (dict(rot=Rotation(FAKE, 10, 80, 0)), 1),
    (dict(rot=Rotation(None, 10, 64, 0)), 1), (dict(tokens=1 << 29), 2),
    (dict(tokens=0, k=heads(None), pos=None), 0)])
def test_append_errors(lib, kw, want):  # noqa: F811
    assert append(lib, **kw) == want


def read(lib, c=cache(), k=heads(), v=heads(), tokens=1, pos=FAKE, seq=None,  # noqa: F811
         t=table()):
    lib.w4_kv_read.argtypes = [P, P, P, I, P, P, P, P]
    return lib.w4_kv_read(ref(c), ref(k), ref(v), tokens, pos, seq, ref(t), None)


@pytest.mark.parametrize("kw,want", [
    (dict(c=None), 1), (dict(k=None, v=None), 1), (dict(k=heads(None)), 1),
    (dict(v=heads(FAKE + 2)), 1), (dict(tokens=-2), 1), (dict(pos=None), 1), (dict(t=None), 1),
    (dict(tokens=3, t=table(seqs=2)), 1), (dict(tokens=1 << 30), 2), (dict(tokens=0), 0)])
def test_read_errors(lib, kw, want):  # noqa: F811
    assert read(lib, **kw) == want


def attn(lib, c=cache(), q=heads(), out=heads(), hq=4, tokens=1, lens=FAKE,  # noqa: F811
         t=table(), scale=0.125, window=0, lse=None, ws=FAKE, n=1 << 40, f32=False):
    fn = lib.w4_paged_attn_f32 if f32 else lib.w4_paged_attn
    fn.argtypes = [P, P, P, I, I, P, P, ctypes.c_float, I, P, P, ctypes.c_size_t, P]
    return fn(ref(c), ref(q), ref(out), hq, tokens, lens, ref(t), scale, window, lse, ws, n, None)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(c=None), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(q=heads(None)), 1),
    (dict(out=heads(FAKE + 4)), 1), (dict(q=heads(token=4)), 1), (dict(hq=0), 1),
    (dict(hq=3), 1), (dict(tokens=0), 2), (dict(tokens=9), 2), (dict(lens=None), 1),
    (dict(lens=FAKE + 2), 1), (dict(t=None), 1), (dict(t=table(width=0)), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(window=-1), 1),
    (dict(lse=FAKE + 2), 1), (dict(ws=None), 1), (dict(ws=FAKE + 128), 1),
    (dict(t=table(width=1 << 27, stride=1 << 27)), 2)])
def test_attn_errors(lib, kw, want, f32):  # noqa: F811
    assert attn(lib, f32=f32, **kw) == want


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D", [64, 128])
def test_layout_places_are_distinct(fmt, D):
    """Every value of a record has a place of its own inside it."""
    width = {"bf16": 2, "int8": 1, "int4": 1}[fmt]
    seen = set()
    for which in kv.places(fmt, D):
        for byte, nib in which.reshape(-1, 2):
            seen.add((int(byte), int(nib)))
            assert 0 <= byte and byte + width <= 32 * D * {"bf16": 2, "int8": 1, "int4": 0.5}[fmt]
    assert len(seen) == 32 * D


def test_plain_quantiser_by_hand():
    # range -1..2 in 15 steps of 0.2 (binary16 0.199951): z = 5, 2.0 -> 10 above it
    q, s, z = kv.quantise(np.array([[-1.0, 2.0, 0.0, 0.1]], np.float32), "int4")
    assert s[0] == np.float16(0.2) and z[0] == 5 and q[0].tolist() == [0, 15, 5, 6]
    q, s, z = kv.quantise(np.array([[0.0, 0.0]], np.float32), "int8")
    assert s[0] == 0 and z[0] == 0 and q[0].tolist() == [0, 0]


def test_plain_attention_by_hand():
    q = np.zeros((1, 1, 2), np.float32)
    k = [np.ones((3, 1, 2), np.float32)]
    v = [np.arange(6, dtype=np.float32).reshape(3, 1, 2)]
    out, lse, mag = kv.attention(q, k, v, [3], 1, 1.0, 0)
    assert np.allclose(out, [[[2, 3]]]) and np.allclose(lse, np.log(3)) and np.allclose(mag, out)
    out, lse, _ = kv.attention(q, k, v, [3], 1, 1.0, 2)
    assert np.allclose(out, [[[3, 4]]]) and np.allclose(lse, np.log(2))
    out, lse, _ = kv.attention(q, k, v, [0], 1, 1.0, 0)
    assert (out == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("mistake", ["window", "causal", "scale", "head"])
def test_planted_mistakes_leave_the_bound(mistake):
    """The attention's tolerances catch an oracle that is slightly wrong."""
    rng = np.random.default_rng(0)
    lens, M, H, R, D = [40], 2, 2, 2, 64
    q = rng.standard_normal((M, H * R, D)).astype(np.float32)
    k = [rng.standard_normal((40, H, D)).astype(np.float32)]
    v = [rng.standard_normal((40, H, D)).astype(np.float32)]
    ref = kv.attention(q, k, v, lens, M, 0.125, 20)
    a = dict(q=q, keys=k, values=v, lens=lens, tokens=M, scale=0.125, window=20)
    if mistake == "window":
        a["window"] = 21
    elif mistake == "causal":
        a["lens"], a["keys"], a["values"] = [39], [k[0][:39]], [v[0][:39]]
    elif mistake == "scale":
        a["scale"] = 0.13
    else:
        a["keys"] = [k[0][:, ::-1]]
    bad, bad_lse, _ = kv.attention(**a)
    dS = kv.score_error("bf16", q, k, None, lens, 0.125)
    kv.check_attention(ref[0], ref[1], *ref, "bf16", dS, 40, False)
    with pytest.raises(AssertionError):
        kv.check_attention(bad, bad_lse, *ref, "bf16", dS, 40, False)
