"""The calls for long contexts where their documentation allows more than an
ordinary step asks for: tables much wider than the sequences, many sequences, wide
groups, large pages, first calls of a process under capture, graphs replayed side by
side, one list for lengths and counts."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest

from tests import kv_testutil as kv
from tests.test_gpu_attn_weights import check as check_weights
from tests.test_gpu_key_blocks import run_both as run_blocks
from tests.test_gpu_kv_gather import Moving
from tests.test_gpu_paged_attn import Setup, i32
from tests.test_gpu_sparse_attn import lists, run_both as run_sparse

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def w4():
    from int4_weight_only_w4_gb300 import w4 as mod
    return mod


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_wide_tables(w4, fmt):
    """Room for 20000 pages a sequence, most of it not there: the results of a narrow
    table, bit for bit."""
    lens, P = [300, 0, 17, 1000, 64] * 12, 16
    s = Setup(w4, fmt, 64, 2, 3, P, 2, lens, seed=1)
    B, width = s.table.shape
    wide = torch.full((B, 20000), -7, device="cuda", dtype=torch.int32)
    wide[:, :width] = s.table
    c = s.cache
    bounds = [c.new_bounds() for _ in range(2)]
    scores = [torch.full((B, 2, 20000), 7.0, device="cuda") for _ in range(2)]
    lse = c.attend(s.gq, s.glens, s.table)[1]
    weights = [torch.full((B, 2, 1100), 7.0, device="cuda") for _ in range(2)]
    for table, b, x, w in zip((s.table, wide), bounds, scores, weights):
        c.key_bounds(b, s.glens, table, tokens=10 ** 9)
        c.block_scores(b, s.gq, s.glens, table, scores=x)
        c.attn_weights(s.gq, lse, s.glens, table, weights=w)
    c.check()
    for a, b in (bounds, scores, weights):
        assert torch.equal(a, b)
    index = torch.full((B, 2, 9), -1, device="cuda", dtype=torch.int32)
    counts = torch.zeros(B, device="cuda", dtype=torch.int32)
    w4.select(scores[0], s.glens, index, counts, unit=P, last=1)
    for a, b in zip(c.attend_blocks(s.gq, s.glens, s.table, index, counts),
                    c.attend_blocks(s.gq, s.glens, wide, index, counts)):
        assert torch.equal(a, b)
    m = Moving(w4, fmt, 64, 2, P, lens, 20, seed=2)
    there = [min(n, 20) for n in lens]
    index, pool = i32(m.lists(there)), m.cache.pool.clone()
    m.cache.gather(m.s.table, m.s.glens, index, i32(there), m.to)
    want = m.cache.pool.clone()
    m.cache.pool.copy_(pool)
    wide_from = torch.full((B, 20000), -7, device="cuda", dtype=torch.int32)
    wide_from[:, :m.s.table.shape[1]] = m.s.table
    wide_to = torch.full((B, 20000), -7, device="cuda", dtype=torch.int32)
    wide_to[:, :m.to.shape[1]] = m.to
    m.cache.gather(wide_from, m.s.glens, index, i32(there), wide_to)
    assert torch.equal(m.cache.pool, want)
    m.cache.check()


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_many_short_lists(w4, fmt):
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 60, 700)
    lens[[3, 400, 699]] = [600, 0, 333]
    s = Setup(w4, fmt, 64, 1, 4, 16, 1, lens.tolist(), seed=12)
    run_sparse(w4, s, 16, *lists(rng, s.lens, 1, 16, 4))
    s.cache.check()


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_wide_groups(w4, fmt):
    """100 query heads of one key/value head, 8 new tokens: 800 rows."""
    lens, P = [70, 5, 0, 33], 16
    s = Setup(w4, fmt, 64, 1, 100, P, 8, lens, seed=4)
    run_blocks(w4, s, P, 8, 8)
    run_sparse(w4, s, P, *lists(np.random.default_rng(3), lens, 1, P, 3))
    lse = s.cache.attend(s.gq, s.glens, s.table)[1]
    before = torch.rand(4, 1, 80, device="cuda")
    got = torch.full((4, 1, 80), 7.0, device="cuda")
    s.cache.attn_weights(s.gq, lse, s.glens, s.table, before=before, decay=0.5, weights=got)
    check_weights(s, got.cpu().numpy(), lse.cpu().numpy(), before=before.cpu().numpy(), decay=0.5)
    s.cache.check()


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_large_pages(w4, fmt):
    lens, P = [3000, 1, 1024, 1025, 0], 1024
    s = Setup(w4, fmt, 64, 2, 2, P, 2, lens, seed=6, spare=0)
    run_blocks(w4, s, P, 1500, 2)
    run_sparse(w4, s, P, *lists(np.random.default_rng(3), lens, 2, P, 2))
    m = Moving(w4, fmt, 64, 2, P, lens, 1100, seed=7)
    counts = [1100, 1, 1000, 17, 0]
    m.check(m.lists(counts), counts)
    s.cache.check()


def test_counts_are_the_new_lengths(w4):
    """Selection and moving write and read the lengths' own kind of list; the call after
    them reads it on the device."""
    m = Moving(w4, "int8", 64, 2, 16, [400, 30, 0], 64, seed=8)
    score = torch.rand(3, 2, 400, device="cuda")
    index = torch.zeros(3, 2, 50, device="cuda", dtype=torch.int32)
    lens = m.s.glens.clone()
    w4.select(score, m.s.glens, index, lens, last=5)
    m.cache.gather(m.s.table, m.s.glens, index, lens, m.to)
    w = torch.rand(3, 2, 400, device="cuda")
    out = m.cache.gather(m.s.table, m.s.glens, index, lens, m.to, weights=w)
    assert lens.tolist() == [50, 30, 0]
    for b, n in enumerate(lens.tolist()):
        assert torch.equal(out[b, :, :n], w[b].gather(1, index[b, :, :n].long()))
        assert (out[b, :, n:] == 0).all() and out.shape == w.shape
    m.cache.check()


@pytest.mark.parametrize("draft", [1, 3])
def test_a_layer_over_selected_blocks(draft):
    """The example's layer: with as many blocks as there are it is the whole layer up to
    the order of sums; with few it runs."""
    spec = importlib.util.spec_from_file_location(
        "decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    ex = sys.modules[spec.name] = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    whole, _ = ex.run("0.5b", "bf16", seqs=2, prompt=90, steps=6, draft=draft)
    all_blocks, _ = ex.run("0.5b", "bf16", seqs=2, prompt=90, steps=6, draft=draft, blocks=6)
    few, _ = ex.run("0.5b", "bf16", seqs=2, prompt=90, steps=6, draft=draft, blocks=3)
    # the attention's outputs differ by a rounding to bf16 that falls the other way, 2^-8
    # of a value at most and of few values; the products after it keep its size or less
    # beside the residual sum
    off = (all_blocks.float() - whole.float()).norm() / whole.float().norm()
    assert off <= 2.0 ** -8
    assert torch.isfinite(few.float()).all()
    assert torch.equal(few[:, :48], all_blocks[:, :48])    # three blocks: all of them


def _all_calls(w4):
    """A cache with six sequences, and a function that makes every call on it."""
    lens, P, B, H = [900, 1, 0, 333, 64, 2000], 16, 6, 2
    s = Setup(w4, "int8", 64, H, 3, P, 2, lens, seed=9)
    c, width = s.cache, s.table.shape[1]
    d = dict(device="cuda")
    out = dict(bounds=c.new_bounds(), scores=torch.zeros(B, H, width, **d),
               index=torch.zeros(B, H, 8, dtype=torch.int32, **d),
               counts=torch.zeros(B, dtype=torch.int32, **d), out=torch.empty_like(s.gq),
               lse=torch.empty(s.gq.shape[:2], **d), weights=torch.zeros(B, H, 2000, **d),
               kept=torch.zeros(B, H, 40, dtype=torch.int32, **d),
               lens=torch.zeros(B, dtype=torch.int32, **d),
               moved=torch.zeros(B, H, 40, **d))
    big = w4.PagedCache(torch.cat([c.pool, c.pool]), w4.KV_INT8, H, 64, P)
    to = torch.arange(B * 3, dtype=torch.int32, **d).view(B, 3) + c.pages

    def calls(ws):
        o = out
        c.key_bounds(o["bounds"], s.glens, s.table, tokens=5000)
        c.block_scores(o["bounds"], s.gq, s.glens, s.table, scores=o["scores"])
        w4.select(o["scores"], s.glens, o["index"], o["counts"], unit=P, last=1)
        c.attend_blocks(s.gq, s.glens, s.table, o["index"], o["counts"], out=o["out"],
                        lse=o["lse"], workspace=ws)
        c.attn_weights(s.gq, o["lse"], s.glens, s.table, weights=o["weights"])
        w4.select(o["weights"], s.glens, o["kept"], o["lens"], first=1, last=4)
        big.gather(s.table, s.glens, o["kept"], o["lens"], to, weights=o["weights"],
                   weights_out=o["moved"])
    out["pool"] = big.pool
    return c, calls, out


def test_graphs_side_by_side(w4):
    """Two graphs of all calls, replayed on two streams at once, and eager calls beside
    them: the results of the calls alone."""
    sets = [_all_calls(w4) for _ in range(3)]
    wants, graphs = [], []
    for c, calls, out in sets:
        calls(c.new_workspace())
        torch.cuda.synchronize()
        wants.append({k: v.clone() for k, v in out.items()})
    for c, calls, out in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls(None)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        torch.cuda.synchronize()
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        sets[2][1](None)
    torch.cuda.synchronize()
    for (c, _, out), want in zip(sets, wants):
        c.check()
        for k, v in out.items():
            assert torch.equal(v, want[k]), k


def first_calls_captured():
    """All calls, the first ones of a process, under capture; then eager ones."""
    from int4_weight_only_w4_gb300 import w4
    c, calls, out = _all_calls(w4)
    ws = torch.empty(w4.paged_attn_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(ws)
    graph.replay()
    torch.cuda.synchronize()
    got = {k: v.clone() for k, v in out.items()}
    for v in out.values():
        if v is not out["pool"]:
            v.zero_()
    calls(ws)
    torch.cuda.synchronize()
    c.check()
    for k, v in out.items():
        assert torch.equal(v, got[k]), k
    print("captured first")


def test_first_calls_of_a_process_captured():
    code = "from tests.test_gpu_long_edges import first_calls_captured as f; f()"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=240)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
