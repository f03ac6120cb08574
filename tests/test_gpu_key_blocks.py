"""w4_key_bounds and w4_block_scores against the values that the cache holds:
formats, head layouts, page sizes, lengths of zero, one and around every border,
new tokens from one to a whole prompt, values that are not finite, strides, other
streams, graphs, offsets past 32 bits, what is to stay as it is, refusals.

Bounds are exact.  A score is a sum of 2 D products of bfloat16 values (each exact
in fp32) with 2 D fp32 additions: off by at most (2 D + 4) 2^-23 of the sum of the
products' magnitudes."""
import numpy as np
import pytest

from tests import kv_testutil as kv
from tests.test_gpu_paged_attn import Setup, i32, to_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500]
MARK = 7.0


@pytest.fixture(scope="module")
def w4():
    from int4_weight_only_w4_gb300 import w4 as mod
    return mod


def host(t):
    return t.float().cpu().numpy()


def marked_bounds(s):
    return torch.full(s.cache.bounds_shape, MARK, device="cuda", dtype=torch.bfloat16)


def want_bounds(s, tokens, P):
    """[pages, heads, 2, D]; MARK where nothing is written."""
    pages, H, _, D = s.cache.bounds_shape
    out = np.full((pages, H, 2, D), MARK, np.float32)
    table = s.table.cpu().numpy()
    for b, n in enumerate(s.lens):
        if n <= 0:
            continue
        k = kv.bf16(s.keys[b])
        for i in range(max(0, n - tokens) // P, (n - 1) // P + 1):
            part = k[i * P:min(n, i * P + P)]
            out[table[b, i], :, 0], out[table[b, i], :, 1] = part.max(0), part.min(0)
    return out


def want_scores(bounds, q, lens, tokens, table, P, H, columns):
    """(scores [B, H, columns], sum of magnitudes of the one that counts); MARK past
    the blocks."""
    B, (T, HQ, D) = len(lens), q.shape
    out = np.full((B, H, columns), MARK)
    mag = np.zeros((B, H, columns))
    G = HQ // H
    for b, n in enumerate(lens):
        first = max(0, tokens - n)
        rows = q[b * tokens + first:(b + 1) * tokens].astype(np.float64)
        for i in range(-(-max(n, 0) // P)):
            hi, lo = bounds[table[b, i]].astype(np.float64).transpose(1, 0, 2)
            for h in range(H):
                x = rows[:, h * G:(h + 1) * G].reshape(-1, D)
                terms = np.where(x >= 0, x * hi[h], x * lo[h])
                out[b, h, i] = terms.sum(-1).max()
                mag[b, h, i] = np.abs(terms).sum(-1).max()
    return out, mag


def check_scores(got, want, mag, D, what=""):
    err = np.abs(got.astype(np.float64) - want)
    assert (err <= (2 * D + 4) * 2.0 ** -23 * mag).all(), (what, float(err.max()))


def run_both(w4, s, P, tokens, score_tokens):
    bounds = marked_bounds(s)
    s.cache.key_bounds(bounds, s.glens, s.table, tokens=tokens)
    assert np.array_equal(host(bounds), want_bounds(s, tokens, P))
    s.cache.key_bounds(bounds, s.glens, s.table, tokens=10 ** 6)
    full = host(bounds)
    assert np.array_equal(full, want_bounds(s, 10 ** 6, P))
    H, D = s.cache.kv_heads, s.cache.head_dim
    columns = s.table.shape[1] + 3
    scores = torch.full((len(s.lens), H, columns), MARK, device="cuda")
    w4.block_scores(s.cache, bounds, s.gq, s.glens, s.table, scores)
    want, mag = want_scores(full, s.q, s.lens, score_tokens, s.table.cpu().numpy(), P, H, columns)
    check_scores(host(scores), want, mag, D)
    s.cache.check()
    return bounds, scores


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D,H,group,P", [(128, 4, 7, 16), (64, 2, 7, 32), (128, 1, 1, 64),
                                         (64, 3, 5, 16), (128, 2, 8, 48), (64, 1, 12, 16),
                                         (128, 1, 33, 128)])
@pytest.mark.parametrize("M", [1, 3, 8])
def test_formats_and_heads(w4, fmt, D, H, group, P, M):
    run_both(w4, Setup(w4, fmt, D, H, group, P, M, LENS[M % 2::2], seed=D + H + group + M), P,
             M, M)


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 33, 64, 100, 2000])
def test_new_tokens(w4, tokens):
    s = Setup(w4, "int8", 64, 2, 3, 32, 2, [0, 1, 31, 32, 33, 64, 65, 333, 1000], seed=tokens)
    run_both(w4, s, 32, tokens, 2)


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_many_sequences(w4, fmt):
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 40, 700)
    lens[[3, 400, 699]] = [600, 0, 333]
    run_both(w4, Setup(w4, fmt, 64, 1, 4, 16, 1, lens.tolist(), seed=2), 16, 1, 1)


@pytest.mark.parametrize("lens", [[0], [1], [5, 0], [0, 0, 0], [0, 0, 900, 0], [3000]])
def test_lengths(w4, lens):
    run_both(w4, Setup(w4, "bf16", 128, 2, 3, 16, 5, lens, seed=len(lens)), 16, 5, 5)


def test_values_that_are_not_finite(w4):
    """NaN among a block's keys makes its bounds NaN, and its score infinite; an
    infinity is a bound, and its block's score infinite too; others do not change."""
    n, P = 100, 16
    s = Setup(w4, "bf16", 64, 2, 2, P, 1, [n], seed=5)
    bounds, scores = run_both(w4, s, P, n, 1)
    clean, before = host(bounds), host(scores)
    k, v = s.keys[0].copy(), s.values[0]
    k[20, 0, 3], k[40, 1, 5], k[41, 1, 6] = np.nan, np.inf, -np.inf
    s.cache.append(to_gpu(k), to_gpu(v), i32(np.arange(n)), s.table)
    s.cache.key_bounds(bounds, s.glens, s.table, tokens=n)
    w4.block_scores(s.cache, bounds, s.gq, s.glens, s.table, scores)
    got, table = host(bounds), s.table[0].cpu().numpy()
    assert np.isnan(got[table[1], 0, :, 3]).all()
    assert got[table[2], 1, 0, 5] == np.inf and got[table[2], 1, 1, 6] == -np.inf
    same = np.ones(got.shape, bool)
    same[table[1], 0, :, 3] = same[table[2], 1, 0, 5] = same[table[2], 1, 1, 6] = False
    assert np.array_equal(got[same], clean[same])
    after, change = host(scores), np.zeros(before.shape, bool)
    change[0, 0, 1] = change[0, 1, 2] = True
    assert np.isposinf(after[change]).all() and np.array_equal(after[~change], before[~change])
    # a query that is not finite: every block of its head
    q = s.gq.clone()
    q[0, 0, 9] = float("nan")
    w4.block_scores(s.cache, bounds, q, s.glens, s.table, scores)
    assert np.isposinf(host(scores)[0, 0, :7]).all()
    assert np.array_equal(host(scores)[0, 1], after[0, 1])


def test_queries_of_any_size(w4):
    """Scores scale with the queries, exactly, until they leave fp32."""
    s = Setup(w4, "bf16", 128, 2, 3, 16, 2, [100, 33], seed=7)
    bounds, scores = run_both(w4, s, 16, 100, 2)
    for power in (-60, 60):
        got = torch.full_like(scores, MARK)
        w4.block_scores(s.cache, bounds, s.gq * 2.0 ** power, s.glens, s.table, got)
        there = scores != MARK
        assert torch.equal(got[there], scores[there] * 2.0 ** power)
    w4.block_scores(s.cache, bounds * 1e30, s.gq * 1e30, s.glens, s.table, got)
    assert torch.isposinf(got[there]).all()


def test_bad_pages_and_lengths_are_recorded(w4):
    s = Setup(w4, "int8", 64, 2, 2, 16, 1, [40, 50], seed=8)
    table = s.table.clone()
    table[0, 1], table[1, 2] = 10 ** 6, -3
    bounds = marked_bounds(s)
    s.cache.key_bounds(bounds, s.glens, table, tokens=100)
    torch.cuda.synchronize()
    assert s.cache.error.item() == w4.KV_ERR_PAGE
    want, pages = want_bounds(s, 100, 16), s.table.cpu().numpy()
    want[pages[0, 1]] = want[pages[1, 2]] = MARK
    assert np.array_equal(host(bounds), want)
    s.cache.error.zero_()
    scores = torch.full((2, 2, table.shape[1]), MARK, device="cuda")
    w4.block_scores(s.cache, bounds, s.gq, s.glens, table, scores)
    torch.cuda.synchronize()
    assert s.cache.error.item() == w4.KV_ERR_PAGE
    got = host(scores)
    assert np.isneginf(got[0, :, 1]).all() and np.isneginf(got[1, :, 2]).all()
    assert np.isfinite(got[0, :, [0, 2]]).all() and (got[0, :, 3:] == MARK).all()
    for call in (lambda t: s.cache.key_bounds(bounds, i32([40, 50]), t, tokens=100),
                 lambda t: s.cache.block_scores(bounds, s.gq, i32([40, 50]), t)):
        s.cache.error.zero_()
        call(s.table[:, :3].contiguous())                   # room for 48 tokens
        torch.cuda.synchronize()
        assert s.cache.error.item() == w4.KV_ERR_LENGTH
    s.cache.error.zero_()
    bounds.fill_(MARK)
    s.cache.key_bounds(bounds, i32([-5, -1]), s.table, tokens=100)
    assert (bounds == MARK).all()
    s.cache.check()


def test_strides_stream_graph_and_repeats(w4):
    s = Setup(w4, "int4", 128, 2, 7, 16, 3, [100, 1, 700, 0], seed=3)
    bounds, scores = run_both(w4, s, 16, 3, 3)
    T, HQ, D = s.q.shape
    rows = torch.zeros(T, HQ + 4, D, device="cuda", dtype=torch.bfloat16)
    rows[:, 1:HQ + 1] = s.gq
    got = torch.full_like(scores, MARK)
    w4.block_scores(s.cache, bounds, rows[:, 1:HQ + 1], s.glens, s.table, got)
    assert torch.equal(got, scores)
    wide = torch.full((4, 2 * s.table.shape[1]), -7, device="cuda", dtype=torch.int32)
    wide[:, :s.table.shape[1]] = s.table
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = marked_bounds(s)
    got = s.cache.block_scores(s.cache.key_bounds(other, s.glens, wide[:, :s.table.shape[1]],
                                                  tokens=1000, stream=side),
                               s.gq, s.glens, s.table, stream=side)
    side.synchronize()
    assert torch.equal(other, bounds)
    there = got > -torch.inf
    assert torch.equal(got[there], scores[..., :got.shape[2]][there])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.key_bounds(other, s.glens, s.table, tokens=1000)
        s.cache.block_scores(other, s.gq, s.glens, s.table, scores=got)
    for _ in range(3):
        other.fill_(MARK)
        got.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(other, bounds)
        assert torch.equal(got, scores[..., :got.shape[2]])


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_offsets_past_32_bits(w4, fmt):
    H, D, P = 4, 128, 16
    per_page = w4.kv_pool_bytes(kv.FMT[fmt], H, D, P, 1)
    pages = max((5 << 30) // per_page, (5 << 30) // (4 * H * D))
    if torch.cuda.mem_get_info()[0] < pages * per_page + (8 << 30):
        pytest.skip("needs more memory")
    s = Setup(w4, fmt, D, H, 2, P, 1, [33], seed=13)
    cache = w4.PagedCache(torch.empty(pages * per_page, dtype=torch.uint8, device="cuda"),
                          kv.FMT[fmt], H, D, P)
    table = i32([[pages - 1, 5, pages // 2 + 3]])
    for a, b in zip(s.table[0, :3].tolist(), table[0].tolist()):
        cache.pool.view(-1, per_page)[b] = s.cache.pool.view(-1, per_page)[a]
    bounds = torch.empty(cache.bounds_shape, device="cuda", dtype=torch.bfloat16)
    cache.key_bounds(bounds, s.glens, table, tokens=33)
    small = marked_bounds(s)
    s.cache.key_bounds(small, s.glens, s.table, tokens=33)
    assert torch.equal(bounds[table[0].long()], small[s.table[0, :3].long()])
    assert torch.equal(cache.block_scores(bounds, s.gq, s.glens, table),
                       s.cache.block_scores(small, s.gq, s.glens, s.table)[..., :3])
    cache.check()


def test_refusals(w4):
    s = Setup(w4, "int4", 64, 2, 2, 16, 1, [5, 6], seed=1)
    bounds, c = s.cache.new_bounds(), s.cache
    c.key_bounds(bounds, s.glens, s.table)

    def status(f, *args, **kw):
        with pytest.raises(w4.W4Error) as e:
            f(*args, **kw)
        return e.value.status

    for bad in (bounds[:-1], bounds.float(), bounds.cpu(), bounds.transpose(0, 1)):
        with pytest.raises(ValueError):
            c.key_bounds(bad, s.glens, s.table)
        with pytest.raises(ValueError):
            c.block_scores(bad, s.gq, s.glens, s.table)
    with pytest.raises(ValueError):
        c.key_bounds(bounds, s.glens[:1], s.table)
    assert status(c.key_bounds, bounds, s.glens, s.table, tokens=0) == w4.Status.INVALID_ARG
    for q in (s.gq[:1], s.gq[..., :32], s.gq.float()):
        with pytest.raises(ValueError):
            c.block_scores(bounds, q, s.glens, s.table)
    with pytest.raises(ValueError):
        c.block_scores(bounds, s.gq, s.glens, s.table,
                       scores=torch.zeros(2, 3, 9, device="cuda"))
    width = s.table.shape[1]
    assert status(c.block_scores, bounds, s.gq, s.glens, s.table,
                  scores=torch.zeros(2, 2, width - 1, device="cuda")) == w4.Status.INVALID_ARG
    assert status(c.block_scores, bounds, s.gq[:, :3], s.glens, s.table) == w4.Status.INVALID_ARG
    nine = torch.zeros(18, 4, 64, device="cuda", dtype=torch.bfloat16)
    assert status(c.block_scores, bounds, nine, s.glens, s.table) == w4.Status.UNSUPPORTED
    odd = torch.zeros(2 * 4 * 64 + 4, device="cuda", dtype=torch.bfloat16)[4:].view(2, 4, 64)
    assert status(c.block_scores, bounds, odd, s.glens, s.table) == w4.Status.INVALID_ARG
