"""w4_attn_weights against fp64 over the keys that the cache holds: formats, head
layouts (also more rows than a block of the device holds at once), 1-8 new tokens,
lengths around every border, windows, decays, weights in place, what lies past the
length, rows without keys, streams, graphs, offsets past 32 bits, refusals.

A probability is exp of (score - lse): its relative error is at most that of the
exponent, dS of kv_testutil for the score's sum and 2^-22 (|score| + |lse| + 4) for
the products, the difference and the two logarithms' conversions, plus 2^-21 for
exp2 and (rows + 8) 2^-23 for the sum; numbers under 2^-126 become 0."""
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


def reference(s, lse, scale, window, before, decay, columns):
    """Weights, what the new tokens add to them, and the exponents' largest parts."""
    T, HQ, D = s.q.shape
    H, M = s.cache.kv_heads, s.M
    G = HQ // H
    out, add = np.full((len(s.lens), H, columns), MARK), np.zeros((len(s.lens), H, columns))
    most = 0.0
    for b, n in enumerate(s.lens):
        if n <= 0:
            continue
        j = np.arange(n)
        for h in range(H):
            k = s.keys[b][:, h].astype(np.float64)
            total = np.zeros(n)
            for i in range(M):
                last = n - M + i
                seen = (j <= last) & ((j > last - window) if window else True)
                for g in range(h * G, (h + 1) * G):
                    e = lse[b * M + i, g]
                    if not np.isfinite(e) or not seen.any():
                        continue
                    x = k @ s.q[b * M + i, g].astype(np.float64) * scale
                    total += np.where(seen, np.exp(np.minimum(x - e, 80)), 0)
                    most = max(most, np.abs(x[seen]).max() + abs(float(e)))
            add[b, h, :n] = total
            out[b, h, :n] = total
            old = max(0, n - M)
            if before is not None:
                out[b, h, :old] += decay * before[b, h, :old].astype(np.float64)
    return out, add, most


def check(s, got, lse, scale=None, window=0, before=None, decay=1.0, what=""):
    D = s.q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    columns = got.shape[2]
    want, add, most = reference(s, lse, scale, window, before, decay, columns)
    dS = kv.score_error(s.fmt, s.q, s.keys, s.scales, s.lens, scale)
    rows = s.M * (s.q.shape[1] // s.cache.kv_heads)
    u = dS + 2.0 ** -22 * (most + 4) + 2.0 ** -21 + (rows + 8) * 2.0 ** -23
    err = np.abs(got.astype(np.float64) - want)
    bound = u * add + 2.0 ** -22 * np.abs(want) + 1e-37 * rows
    there = np.zeros(want.shape, bool)
    for b, n in enumerate(s.lens):
        there[b, :, :max(n, 0)] = True
    assert (got[~there] == MARK).all(), what
    assert (err[there] <= bound[there]).all(), (what, float((err / bound)[there].max()))


def attend(s, scale=None, window=0):
    return s.cache.attend(s.gq, s.glens, s.table, scale=scale, window=window)[1]


def run(w4, s, scale=None, window=0, decay=0.75, spare=5):
    """From nothing, from other weights, and in place."""
    B, H = len(s.lens), s.cache.kv_heads
    columns = max(max(s.lens), 1) + spare
    lse = attend(s, scale, window)
    host = lse.cpu().numpy()
    new = lambda: torch.full((B, H, columns), MARK, device="cuda")  # noqa: E731
    got = new()
    w4.attn_weights(s.cache, s.gq, lse, s.glens, s.table, got, scale=scale, window=window)
    check(s, got.cpu().numpy(), host, scale, window, what="alone")
    rng = np.random.default_rng(columns)
    old = np.exp(2 * rng.standard_normal((B, H, columns))).astype(np.float32)
    before = torch.from_numpy(old).cuda()
    got = new()
    kw = dict(before=before, decay=decay, scale=scale, window=window)
    w4.attn_weights(s.cache, s.gq, lse, s.glens, s.table, got, **kw)
    check(s, got.cpu().numpy(), host, scale, window, old, decay, what="added")
    placed = before.clone()
    w4.attn_weights(s.cache, s.gq, lse, s.glens, s.table, placed, **dict(kw, before=placed))
    for b, n in enumerate(s.lens):
        n = max(n, 0)
        assert torch.equal(placed[b, :, :n], got[b, :, :n])
        assert torch.equal(placed[b, :, n:], before[b, :, n:])
    s.cache.check()
    return got, lse, before


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D,H,group,P", [(128, 4, 7, 16), (64, 2, 7, 32), (128, 1, 1, 64),
                                         (64, 3, 5, 16), (128, 2, 8, 48), (64, 1, 12, 16),
                                         (128, 1, 33, 16)])
@pytest.mark.parametrize("M", [1, 3, 8])
def test_formats_and_heads(w4, fmt, D, H, group, P, M):
    run(w4, Setup(w4, fmt, D, H, group, P, M, LENS[M % 2::2], seed=D + H + group + M))


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("lens", [[0], [1], [5, 0], [0, 0, 0, 0], [16], [700], [3000], [1100, 7],
                                  [2, 1500, 0, 900, 16, 33, 1]])
def test_lengths(w4, fmt, lens):
    for M in (1, 5):
        run(w4, Setup(w4, fmt, 64, 2, 3, 16, M, lens, seed=len(lens) + M))


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 4000])
def test_windows(w4, fmt, window):
    s = Setup(w4, fmt, 128, 2, 4, 32, 4, [0, 1, 3, 16, 19, 100, 117, 333, 900], seed=window)
    run(w4, s, window=window)


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 1e-4])
def test_scales(w4, fmt, scale):
    run(w4, Setup(w4, fmt, 128, 1, 7, 16, 2, [1, 70, 350], seed=9), scale=scale)


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_many_sequences(w4, fmt):
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 40, 700)
    lens[[3, 400, 699]] = [600, 0, 333]
    run(w4, Setup(w4, fmt, 64, 1, 4, 16, 1, lens.tolist(), seed=12))


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("M", [1, 8])
def test_each_row_adds_one(w4, fmt, M):
    lens = [2000, 40, 7, 333]
    s = Setup(w4, fmt, 128, 2, 7, 16, M, lens, seed=M)
    w = s.cache.attn_weights(s.gq, attend(s), s.glens, s.table)
    total = w.double().sum(-1).cpu().numpy()
    for b, n in enumerate(lens):
        want = 7 * min(M, n)                              # rows that see a key
        assert np.allclose(total[b], want, rtol=1e-4)


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("power", [-60, 60])
def test_queries_of_any_size(w4, fmt, power):
    """Queries times a power of two with the scale divided by it: the same bits."""
    s = Setup(w4, fmt, 64, 2, 7, 16, 2, [70, 33], seed=11)
    lse = attend(s)
    want = s.cache.attn_weights(s.gq, lse, s.glens, s.table)
    got = s.cache.attn_weights(s.gq * 2.0 ** power, lse, s.glens, s.table,
                               scale=64 ** -0.5 * 2.0 ** -power)
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_keys_of_zero(w4, fmt):
    """All scores are 0 whatever the queries are: every key of 50 gets 4 / 50."""
    s = Setup(w4, fmt, 128, 1, 4, 16, 1, [50], seed=12, spread=0.0)
    q = torch.full_like(s.gq, 1e35)
    got = s.cache.attn_weights(q, s.cache.attend(q, s.glens, s.table)[1], s.glens, s.table)
    # exp(-ln 50): the logarithm's rounding, 2^-22 of ln 50, and exp2's
    assert (got[0, 0, :50] * 50 / 4 - 1).abs().max() <= 2.0 ** -19


def test_decay_of_zero_reads_nothing(w4):
    s = Setup(w4, "int8", 64, 2, 2, 16, 2, [50, 20], seed=4)
    lse = attend(s)
    nan = torch.full((2, 2, 60), float("nan"), device="cuda")
    want = torch.full((2, 2, 60), MARK, device="cuda")
    w4.attn_weights(s.cache, s.gq, lse, s.glens, s.table, want)
    got = want.clone()
    w4.attn_weights(s.cache, s.gq, lse, s.glens, s.table, got, before=nan, decay=0.0)
    assert torch.equal(got, want)
    # the new tokens' places start anew
    w4.attn_weights(s.cache, s.gq, lse, s.glens, s.table, got, before=nan, decay=0.5)
    for b, n in enumerate(s.lens):
        assert torch.isnan(got[b, :, :n - 2]).all()
        assert torch.equal(got[b, :, n - 2:n], want[b, :, n - 2:n])


def test_rows_and_keys_that_do_not_count(w4):
    """Rows with an infinite log-sum-exp, keys past a row's position that are not
    finite, a page that is not in the pool."""
    M, n = 4, 50
    s = Setup(w4, "bf16", 64, 1, 2, 16, M, [n], seed=5)
    lse = attend(s)
    want = s.cache.attn_weights(s.gq, lse, s.glens, s.table)
    for value in (float("inf"), -float("inf")):
        part = lse.clone()
        part[1, 0] = value
        got = torch.full((1, 1, n), MARK, device="cuda")
        w4.attn_weights(s.cache, s.gq, part, s.glens, s.table, got)
        check(s, got.cpu().numpy(), part.cpu().numpy())
    k = s.keys[0].copy()
    k[n - 1] = np.nan                                     # seen by the last row alone
    s.cache.append(to_gpu(k), to_gpu(s.values[0]), i32(np.arange(n)), s.table)
    got = s.cache.attn_weights(s.gq, lse, s.glens, s.table)
    assert torch.equal(got[..., :n - 1], want[..., :n - 1]) and torch.isnan(got[..., n - 1]).all()
    table = s.table.clone()
    table[0, 1] = 10 ** 6
    got = s.cache.attn_weights(s.gq, lse, s.glens, table)
    torch.cuda.synchronize()
    assert s.cache.error.item() == w4.KV_ERR_PAGE
    assert (got[..., 16:32] == 0).all() and torch.equal(got[..., :16], want[..., :16])
    s.cache.error.zero_()
    short = torch.full((1, 1, 40), MARK, device="cuda")
    w4.attn_weights(s.cache, s.gq, lse, s.glens, s.table, short)
    torch.cuda.synchronize()
    assert s.cache.error.item() == w4.KV_ERR_LENGTH
    s.cache.error.zero_()
    short.fill_(MARK)
    w4.attn_weights(s.cache, s.gq, lse, i32([-1]), s.table, short)
    assert (short == MARK).all()
    s.cache.check()


def test_strides_stream_graph_and_repeats(w4):
    s = Setup(w4, "int4", 128, 2, 7, 16, 3, [100, 1, 700, 0], seed=3)
    want, lse, before = run(w4, s, decay=0.5)
    T, HQ, D = s.q.shape
    rows = torch.zeros(T, HQ + 4, D, device="cuda", dtype=torch.bfloat16)
    rows[:, 1:HQ + 1] = s.gq
    call = lambda q, out, **kw: s.cache.attn_weights(  # noqa: E731
        q, lse, s.glens, s.table, before=before, decay=0.5, weights=out, **kw)
    fresh = lambda: torch.full_like(want, MARK)  # noqa: E731
    assert torch.equal(call(rows[:, 1:HQ + 1], fresh()), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fresh()
    for _ in range(20):
        assert torch.equal(call(s.gq, fresh()), want)
        call(s.gq, other, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    out = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s.gq, out)
    for _ in range(3):
        out.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_offsets_past_32_bits(w4, fmt):
    H, D, P = 4, 128, 16
    per_page = w4.kv_pool_bytes(kv.FMT[fmt], H, D, P, 1)
    pages = (5 << 30) // per_page
    if torch.cuda.mem_get_info()[0] < (7 << 30):
        pytest.skip("needs 7 GB")
    s = Setup(w4, fmt, D, H, 2, P, 1, [33], seed=13)
    cache = w4.PagedCache(torch.empty(pages * per_page, dtype=torch.uint8, device="cuda"),
                          kv.FMT[fmt], H, D, P)
    table = i32([[pages - 1, 5, pages // 2 + 3]])
    for a, b in zip(s.table[0, :3].tolist(), table[0].tolist()):
        cache.pool.view(-1, per_page)[b] = s.cache.pool.view(-1, per_page)[a]
    s.cache, s.table = cache, table
    run(w4, s, spare=1)


def test_refusals(w4):
    s = Setup(w4, "int4", 64, 2, 2, 16, 1, [5, 6], seed=1)
    lse, out = attend(s), torch.zeros(2, 2, 9, device="cuda")
    call = lambda q=s.gq, l=lse, n=s.glens, w=out, **kw: w4.attn_weights(  # noqa: E731
        s.cache, q, l, n, s.table, w, **kw)
    call()
    for kw in (dict(q=s.gq[:1]), dict(q=s.gq.float()), dict(l=lse[:1]), dict(l=lse.double()),
               dict(l=lse[:, :3]), dict(n=s.glens[:1]), dict(w=out[0]), dict(w=out[:1]),
               dict(w=out.half()), dict(w=out[..., :4]), dict(before=out[:, :1]),
               dict(before=out[..., :4].contiguous()), dict(w=out.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(window=-1), dict(scale=float("nan")), dict(decay=float("inf"))):
        with pytest.raises(w4.W4Error) as e:
            call(**kw)
        assert e.value.status == w4.Status.INVALID_ARG
    nine = torch.zeros(18, 4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(w4.W4Error) as e:
        call(q=nine, l=torch.zeros(18, 4, device="cuda"))
    assert e.value.status == w4.Status.UNSUPPORTED
