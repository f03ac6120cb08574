"""The paged attention's division of its work, walked on the host with the
kernel's own arithmetic: over many batches and head layouts, no block leaves
the batch, every record is taken by one block once, and the pieces that are to
be joined are the ones that were written."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests import kv_testutil as kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int4_weight_only_w4_gb300", "csrc")

# (head_dim, kv heads, query heads a kv head) of the library's shapes and others
HEADS = [(128, 4, 7), (64, 2, 7), (128, 8, 4), (64, 8, 1), (128, 2, 8), (64, 3, 5), (128, 1, 33),
         (64, 1, 12)]
SMS = [152, 152, 152, 148, 132, 76, 20, 1, 256, 300]


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("division") / "division.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    "-o", so, os.path.join(ROOT, "tests", "attn_division.cpp")], check=True)
    fn = ctypes.CDLL(so).walk
    I = ctypes.c_int  # noqa: E741
    fn.argtypes = [I, I, I, I, I, I, I, ctypes.c_void_p, I, ctypes.c_void_p]

    def call(fmt, heads, tokens, window, lens, sms):
        D, H, group = heads
        lens = np.ascontiguousarray(lens, np.int32)
        return fn(D, kv.record_bytes(fmt, D), group, H, tokens, window, len(lens),
                  lens.ctypes.data, sms, None)
    return call


# Two cuts in one head of 75 records: the first within 20 of the head's start,
# past the middle of what the head costs, the second inside it.
TIGHT = [([3360, 1200], (128, 4, 7), 1), ([1200, 3360, 1200], (128, 4, 7), 1)]


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("lens,heads,tokens", TIGHT)
def test_heads_little_longer_than_what_is_not_cut_off(walk, fmt, lens, heads, tokens):
    assert walk(fmt, heads, tokens, 0, lens, 152) == 0


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 8])
def test_random_batches(walk, fmt, heads, tokens):
    rng = np.random.default_rng(heads[0] + 10 * heads[1] + 100 * heads[2] + tokens)
    for trial in range(250):
        seqs = int(np.exp(rng.uniform(0, np.log(80))))
        top = int(np.exp(rng.uniform(np.log(20), np.log(20000 if seqs < 9 else 6000))))
        lens = rng.integers(0, top + 1, seqs)
        if trial % 5 == 0:
            lens[:] = top
        if trial % 3 == 0:
            lens[rng.random(seqs) < 0.3] = 0
        window = int(rng.choice([0, 0, 0, 1, 300, 1000, 2 ** 31 - 1]))
        sms = SMS[trial % len(SMS)]
        bad = walk(fmt, heads, tokens, window, lens, sms)
        assert bad == 0, (bad, window, sms, lens.tolist())


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("tokens", [1, 2, 8])
def test_every_pair_of_short_lengths(walk, fmt, tokens):
    """Lengths around what a head costs beside its records, two at a time."""
    for heads in HEADS[:3]:
        for a in range(160, 3600, 176):
            for b in range(160, 3600, 272):
                bad = walk(fmt, heads, tokens, 0, [a, b], 152)
                assert bad == 0, (bad, heads, a, b)


def test_long_and_single_sequences(walk):
    for fmt in kv.FMT:
        for heads in HEADS:
            for lens in ([0], [1], [16], [17], [200], [900], [2000], [65536], [131072] * 4,
                         [131072, 0, 1, 16000], [8] * 700):
                for window in (0, 4096):
                    assert walk(fmt, heads, 1, window, lens, 152) == 0, (fmt, heads, lens)
