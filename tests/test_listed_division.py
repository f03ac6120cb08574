"""The division of the attention over listed blocks, walked on the host as that of
the whole attention is: every record is taken once, the pieces that are to be joined
are the ones that were written, and where the joining launch is left out no head is
cut."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests import kv_testutil as kv
from tests.test_attn_division import CSRC, HEADS, ROOT, SMS

SOURCES = {"listed": "listed_division.cpp", "whole": "attn_division.cpp"}


@pytest.fixture(scope="module", params=list(SOURCES))
def walk(request, tmp_path_factory):
    """walk(...) -> (what is wrong, blocks, records that are not cut off)"""
    so = str(tmp_path_factory.mktemp("division") / f"{request.param}.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    "-o", so, os.path.join(ROOT, "tests", SOURCES[request.param])], check=True)
    fn = ctypes.CDLL(so).walk
    I = ctypes.c_int  # noqa: E741
    fn.argtypes = [I, I, I, I, I, I, I, ctypes.c_void_p, I, ctypes.c_void_p]

    def call(fmt, heads, tokens, records, sms=152):
        D, H, group = heads
        lens = 16 * np.ascontiguousarray(records, np.int32)
        shape = (I * 4)()
        return fn(D, kv.record_bytes(fmt, D), group, H, tokens, 0, len(lens), lens.ctypes.data,
                  sms, shape), shape[0], shape[2]
    call.listed = request.param == "listed"
    return call


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("tokens", range(1, 9))
def test_one_sequence_of_every_length(walk, fmt, tokens):
    for heads in HEADS:
        for records in range(0, 321):
            for sms in (152, 20, 256) if records % 8 == 0 else (152,):
                bad = walk(fmt, heads, tokens, [records], sms)[0]
                assert bad == 0, (bad, heads, records, sms)


def test_short_lists_are_cut(walk):
    """One sequence of the decoder shapes in the lengths at which a listed head is cut
    and one of the whole attention is not (so the test above is about both)."""
    for fmt, heads, tokens, records in [
            ("int8", (128, 4, 7), 1, 78), ("int4", (128, 4, 7), 1, 111),
            ("int8", (128, 4, 7), 4, 30), ("bf16", (64, 2, 7), 1, 80),
            ("int4", (64, 2, 7), 1, 143), ("int8", (64, 2, 7), 8, 23)]:
        bad, blocks, least = walk(fmt, heads, tokens, [records])
        assert bad == 0
        cut = blocks > heads[1] and records >= 2 * least
        assert cut == walk.listed, (fmt, heads, tokens, records, blocks, least)


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 8])
def test_random_lists(walk, fmt, heads, tokens):
    rng = np.random.default_rng(heads[0] + 10 * heads[1] + 100 * heads[2] + tokens)
    for trial in range(150):
        seqs = int(np.exp(rng.uniform(0, np.log(80))))
        top = int(np.exp(rng.uniform(np.log(2), np.log(1200 if seqs < 9 else 300))))
        records = rng.integers(0, top + 1, seqs)
        if trial % 5 == 0:
            records[:] = top
        if trial % 3 == 0:
            records[rng.random(seqs) < 0.3] = 0
        sms = SMS[trial % len(SMS)]
        bad = walk(fmt, heads, tokens, records, sms)[0]
        assert bad == 0, (bad, sms, records.tolist())
