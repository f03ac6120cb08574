"""Host-side checks of the calls for long contexts that need no GPU: argument
errors (every call here fails validation, so no pointer is looked at)."""
import ctypes

import pytest

from tests.test_abi_host import FAKE, lib  # noqa: F401
from tests.test_kv_host import I, P, cache, heads, ref, table


def bounds(lib, c=cache(), out=FAKE, tokens=1, lens=FAKE, t=table()):  # noqa: F811
    lib.w4_key_bounds.argtypes = [P, P, I, P, P, P]
    return lib.w4_key_bounds(ref(c), out, tokens, lens, ref(t), None)


def scores(lib, c=cache(), b=FAKE, q=heads(), hq=2, tokens=1, lens=FAKE, t=table(),  # noqa: F811
           out=FAKE, columns=4):
    lib.w4_block_scores.argtypes = [P, P, P, I, I, P, P, P, I, P]
    return lib.w4_block_scores(ref(c), b, ref(q), hq, tokens, lens, ref(t), out, columns, None)


WALK = [(dict(c=None), 1), (dict(c=cache(pool=None)), 1), (dict(c=cache(pool=FAKE + 64)), 1),
        (dict(c=cache(error=FAKE + 1)), 1), (dict(c=cache(format=3)), 1),
        (dict(c=cache(head_dim=96)), 2), (dict(c=cache(page_tokens=24)), 1), (dict(lens=None), 1),
        (dict(lens=FAKE + 2), 1), (dict(t=None), 1), (dict(t=table(None)), 1),
        (dict(t=table(seqs=0)), 1), (dict(t=table(width=0)), 1), (dict(t=table(stride=3)), 1),
        (dict(t=table(width=1 << 27, stride=1 << 27)), 2),
        (dict(t=table(seqs=1 << 30, width=1, stride=1)), 2),
        (dict(t=table(seqs=1 << 28, width=4)), 2)]
QUERIES = [(dict(q=None), 1), (dict(q=heads(None)), 1), (dict(q=heads(FAKE + 2)), 1),
           (dict(q=heads(token=129)), 1), (dict(q=heads(head=60)), 1), (dict(tokens=0), 2),
           (dict(tokens=9), 2), (dict(hq=0), 1), (dict(hq=3), 1), (dict(hq=2 * 4097), 2)]


@pytest.mark.parametrize("kw,want", WALK + [(dict(out=None), 1), (dict(out=FAKE + 8), 1),
                                            (dict(tokens=0), 1), (dict(tokens=-1), 1)])
def test_key_bounds_errors(lib, kw, want):  # noqa: F811
    assert bounds(lib, **kw) == want


@pytest.mark.parametrize("kw,want", WALK + QUERIES + [
    (dict(b=None), 1), (dict(b=FAKE + 8), 1), (dict(out=None), 1), (dict(out=FAKE + 2), 1),
    (dict(columns=3), 1)])
def test_block_scores_errors(lib, kw, want):  # noqa: F811
    kw = dict(kw)
    if kw.get("t") is not None and kw["t"].width > 4:
        kw["columns"] = 1 << 30
    assert scores(lib, **kw) == want


def select(lib, scores=FAKE, seqs=2, heads=2, columns=9, lens=FAKE, unit=1, first=0,  # noqa: F811
           last=0, count=4, index=FAKE, counts=FAKE):
    lib.w4_select.argtypes = [P, I, I, I, P, I, I, I, I, P, P, P]
    return lib.w4_select(scores, seqs, heads, columns, lens, unit, first, last, count, index,
                         counts, None)


@pytest.mark.parametrize("kw,want", [
    (dict(scores=None), 1), (dict(scores=FAKE + 2), 1), (dict(lens=None), 1),
    (dict(lens=FAKE + 1), 1), (dict(index=None), 1), (dict(index=FAKE + 3), 1),
    (dict(counts=None), 1), (dict(counts=FAKE + 2), 1), (dict(seqs=0), 1), (dict(heads=0), 1),
    (dict(columns=0), 1), (dict(unit=0), 1), (dict(first=-1), 1), (dict(last=-1), 1),
    (dict(count=0), 1), (dict(first=3, last=2), 1),
    (dict(first=(1 << 31) - 1, last=(1 << 31) - 1), 1), (dict(seqs=1 << 26), 2),
    (dict(columns=1 << 30), 2)])
def test_select_errors(lib, kw, want):  # noqa: F811
    assert select(lib, **kw) == want


def sparse(lib, c=cache(), q=heads(), out=heads(), hq=2, tokens=1, lens=FAKE,  # noqa: F811
           t=table(), blocks=FAKE, counts=FAKE, most=4, scale=0.125, lse=None, ws=FAKE, nbytes=0,
           name="w4_sparse_attn"):
    f = getattr(lib, name)
    f.argtypes = [P, P, P, I, I, P, P, P, P, I, ctypes.c_float, P, P, ctypes.c_size_t, P]
    return f(ref(c), ref(q), ref(out), hq, tokens, lens, ref(t), blocks, counts, most, scale, lse,
             ws, nbytes, None)


@pytest.mark.parametrize("name", ["w4_sparse_attn", "w4_sparse_attn_f32"])
@pytest.mark.parametrize("kw,want", [k for k in WALK if "t" not in k[0]] + QUERIES + [
    (dict(t=None), 1), (dict(t=table(None)), 1), (dict(t=table(seqs=1 << 28, width=4)), 2),
    (dict(blocks=None), 1), (dict(blocks=FAKE + 2), 1), (dict(counts=None), 1),
    (dict(counts=FAKE + 1), 1), (dict(most=0), 1), (dict(most=(1 << 31) - 1), 2),
    (dict(out=None), 1), (dict(out=heads(None)), 1), (dict(out=heads(FAKE + 2)), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(lse=FAKE + 2), 1),
    (dict(ws=None), 1), (dict(ws=FAKE + 128), 1)])
def test_sparse_attn_errors(lib, kw, want, name):  # noqa: F811
    assert sparse(lib, name=name, **kw) == want


def weights(lib, c=cache(), q=heads(), lse=FAKE, hq=2, tokens=1, lens=FAKE, t=table(),  # noqa: F811
            scale=0.125, window=0, before=None, decay=1.0, out=FAKE, columns=64):
    lib.w4_attn_weights.argtypes = [P, P, P, I, I, P, P, ctypes.c_float, I, P, ctypes.c_float, P,
                                    I, P]
    return lib.w4_attn_weights(ref(c), ref(q), lse, hq, tokens, lens, ref(t), scale, window,
                               before, decay, out, columns, None)


@pytest.mark.parametrize("kw,want", WALK + QUERIES + [
    (dict(lse=None), 1), (dict(lse=FAKE + 2), 1), (dict(out=None), 1), (dict(out=FAKE + 1), 1),
    (dict(before=FAKE + 2), 1), (dict(columns=0), 1), (dict(window=-1), 1),
    (dict(scale=float("nan")), 1), (dict(decay=float("inf")), 1)])
def test_attn_weights_errors(lib, kw, want):  # noqa: F811
    assert weights(lib, **kw) == want


def gather(lib, c=cache(), t=table(), lens=FAKE, index=FAKE, counts=FAKE, most=4,  # noqa: F811
           to=table(FAKE + 64), w=None, columns=0, out=None, columns_out=4):
    lib.w4_kv_gather.argtypes = [P, P, P, P, P, I, P, P, I, P, I, P]
    return lib.w4_kv_gather(ref(c), ref(t), lens, index, counts, most, ref(to), w, columns, out,
                            columns_out, None)


@pytest.mark.parametrize("kw,want", WALK + [
    (dict(index=None), 1), (dict(index=FAKE + 2), 1), (dict(counts=None), 1),
    (dict(counts=FAKE + 3), 1), (dict(most=0), 1), (dict(to=None), 1), (dict(to=table()), 1),
    (dict(to=table(FAKE + 64, seqs=2)), 1), (dict(to=table(FAKE + 66)), 1),
    (dict(to=table(FAKE + 64, width=1 << 27, stride=1 << 27)), 2), (dict(w=FAKE, columns=9), 1),
    (dict(out=FAKE, columns=9), 1), (dict(w=FAKE, out=FAKE, columns=9), 1),
    (dict(w=FAKE, out=FAKE + 64, columns=0), 1),
    (dict(w=FAKE, out=FAKE + 64, columns=9, columns_out=3), 1), (dict(w=FAKE + 2, out=FAKE + 64, columns=9), 1),
    (dict(w=FAKE, out=FAKE + 65, columns=9), 1)])
def test_gather_errors(lib, kw, want):  # noqa: F811
    assert gather(lib, **kw) == want
