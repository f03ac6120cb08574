"""The paged cache and its attention where they are easily wrong."""
import numpy as np
import pytest

from tests import kv_testutil as kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_kv_cache import bits, i32, rows, to_gpu, w4  # noqa: E402, F401
from tests.test_gpu_paged_attn import Setup, run_both  # noqa: E402


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 9, 1 << 20])
def test_windows_wider_than_any_length(w4, fmt, window):  # noqa: F811
    """They leave nothing out, also where a sequence has fewer tokens than are
    new."""
    for M in (1, 8):
        s = Setup(w4, fmt, 64, 2, 3, 16, M, [0, 1, 5, 7, 8, 9, 40], seed=M)
        want, want_lse = run_both(w4, s)
        got, lse = run_both(w4, s, window=window)
        assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("layout", [None, 0, 1])
@pytest.mark.parametrize("D,first,T", [(128, 0, 32), (64, 0, 48), (128, 3, 9), (64, 15, 2),
                                       (128, 0, 4096)])
def test_nan_is_held_as_zero(w4, fmt, layout, D, first, T):  # noqa: F811
    """NaN beside values of both signs, of one sign, beside infinities and in
    every place of a row, in whole records and in parts of them: held as 0, the
    rest of the row as if it were not there."""
    rng = np.random.default_rng(D + T)
    H = 2
    k, v = rows(rng, T, H, D), rows(rng, T, H, D)
    for x in (k, v):
        for t in range(T):
            x[t, t % H, rng.integers(0, D, 1 + t % 3)] = np.nan
        x[0, 1, :4] = [np.nan, 2.0, np.nan, -1.0]
        if T > 4:
            x[2], x[3] = np.abs(x[2]), -np.abs(x[3])
            x[4, 0, 5:7] = [np.inf, np.nan]
    pos = np.arange(first, first + T, dtype=np.int32)
    rope, kr = None, k
    if layout is not None:
        tab = rng.uniform(0.1, 1, (first + T, D // 2, 2)).astype(np.float32)
        rope = w4.RopeTable(torch.from_numpy(tab).cuda(), layout)
        with np.errstate(invalid="ignore"):
            kr = kv.rotate(k, pos, tab, layout)
    cache = w4.PagedCache.make((first + T) // 16 + 1, kv.FMT[fmt], H, D)
    table = torch.arange((first + T) // 16 + 1, dtype=torch.int32, device="cuda").view(1, -1)
    cache.append(to_gpu(k), to_gpu(v), i32(pos), table, rope=rope)
    got = cache.read(i32(pos), table)
    cache.check()
    for x, g in zip((kr, v), got):
        # 0 widens no row's range; an infinite value is held as Q times the
        # largest scale, which is the code of any value that large
        x = np.nan_to_num(np.asarray(x, np.float32), nan=0.0, posinf=3e38, neginf=-3e38)
        assert np.array_equal(bits(g), kv.bf16_bits(kv.held(x, fmt)))


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("T,HQ", [(1, 14), (5, 3), (700, 28)])
def test_queries_without_a_rotation_are_copied(w4, fmt, T, HQ):  # noqa: F811
    rng = np.random.default_rng(T)
    H, D = 2, 64
    k, v, q = rows(rng, T, H, D), rows(rng, T, H, D), rows(rng, T, HQ, D)
    pages = T // 16 + 1
    cache = w4.PagedCache.make(pages, kv.FMT[fmt], H, D)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    pos = np.arange(T, dtype=np.int32)
    if T > 1:
        pos[1] = -1                                            # padding: left out
    wide = torch.full((T, HQ + 1, D), 9.0, device="cuda", dtype=torch.bfloat16)
    gq = to_gpu(q)
    cache.append(to_gpu(k), to_gpu(v), i32(pos), table, q=gq, q_out=wide[:, 1:])
    cache.check()
    there = pos >= 0
    assert np.array_equal(bits(wide[:, 1:])[there], kv.bf16_bits(q)[there])
    assert (wide[:, 0] == 9.0).all() and (wide[:, 1:][torch.from_numpy(~there).cuda()] == 9.0).all()
    # in place there is nothing to do
    before = gq.clone()
    cache.append(to_gpu(k), to_gpu(v), i32(pos), table, q=gq, q_out=gq)
    assert torch.equal(gq, before)
    k2, v2 = cache.read(i32(pos), table)
    assert np.array_equal(bits(v2)[there], kv.bf16_bits(kv.held(v, fmt))[there])
    # q is looked at: its rows have to lie on 16-byte boundaries
    odd = torch.zeros(T * HQ * D + 4, device="cuda", dtype=torch.bfloat16)[4:].view(T, HQ, D)
    with pytest.raises(w4.W4Error):
        cache.append(to_gpu(k), to_gpu(v), i32(pos), table, q=odd, q_out=wide[:, 1:])


def test_block_tables_whose_rows_overlap_are_refused(w4):  # noqa: F811
    """A row stride below the width (the rows of an expanded table): refused by
    every call, before anything is launched."""
    cache = w4.PagedCache.make(4, w4.KV_INT4, 1, 64)
    x = torch.zeros(3, 1, 64, device="cuda", dtype=torch.bfloat16)
    pos, lens = i32([0, 1, 2]), i32([1, 1, 1])
    one = i32([[2, 1]])
    overlapping = i32([0, 1, 2, 3]).as_strided((3, 2), (1, 1))
    for table in (one.expand(3, -1), overlapping):
        with pytest.raises(ValueError):
            cache.append(x, x, pos, table)
        with pytest.raises(ValueError):
            cache.read(pos, table)
        with pytest.raises(ValueError):
            cache.attend(x, lens, table)
    # one row: its stride does not matter; rows further apart than they are wide
    for table in (one.as_strided((1, 2), (0, 1)), one.as_strided((1, 2), (1, 1)),
                  i32(np.arange(9).reshape(3, 3) % 4)[:, :2]):
        n = table.shape[0]
        cache.append(x[:n], x[:n], pos[:n], table)
        cache.attend(x[:n], lens[:n], table)
    cache.check()


def busy(stream):
    """Some milliseconds of work on a stream."""
    x = torch.ones(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(20):
            x = x @ x * 0.0 + 1.0
    return x


@pytest.mark.parametrize("handle", [False, True])
def test_default_outputs_belong_to_the_calls_stream(w4, handle):  # noqa: F811
    """What a call makes by itself is made, and filled, on the stream that the
    call is given, whatever torch's current stream still has to do."""
    rng = np.random.default_rng(3)
    T, H, D = 64, 2, 64
    k, v = rows(rng, T, H, D), rows(rng, T, H, D)
    cache = w4.PagedCache.make(4, w4.KV_INT8, H, D)
    table, pos = i32([[2, 0, 3, 1]]), i32(np.arange(T))
    cache.append(to_gpu(k), to_gpu(v), pos, table)
    rope = w4.RopeTable(torch.rand(T, D // 2, 2, device="cuda"))
    q, lens = to_gpu(k[:8]), i32([T])
    want = cache.read(pos, table), rope.apply(q, pos[:8]), cache.attend(q, lens, table)
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side
    # memory that the current stream still writes to, free for its next tensors
    for _ in range(3):
        keep = busy(torch.cuda.current_stream())
        for n in (T * H * D, 8 * H * D, 8 * H * 2):
            torch.full((n,), 9.0, device="cuda", dtype=torch.bfloat16)
        got = (cache.read(pos, table, stream=given), rope.apply(q, pos[:8], stream=given),
               cache.attend(q, lens, table, stream=given))
        made = w4.RopeTable.make(100, 64, 1e4, stream=given).table
        torch.cuda.synchronize()
        for a, b in ((got[0][0], want[0][0]), (got[0][1], want[0][1]), (got[1], want[1]),
                     (got[2][0], want[2][0]), (got[2][1], want[2][1])):
            assert torch.equal(a, b)
        assert torch.equal(made, w4.RopeTable.make(100, 64, 1e4).table)
        del keep


def test_check_waits_for_calls_on_other_streams(w4):  # noqa: F811
    cache = w4.PagedCache.make(1, w4.KV_INT4, 1, 64)
    k = torch.zeros(1, 1, 64, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    for _ in range(2):
        keep = busy(side)
        cache.append(k, k, i32([16]), i32([[0]]), stream=side)     # past the block table
        with pytest.raises(w4.W4Error):
            cache.check()
        cache.check()                                              # cleared
        del keep


def test_every_stream_and_graph_has_a_workspace_of_its_own(w4):  # noqa: F811
    """attend() without a workspace: calls on two streams, and a replayed graph
    beside either, share nothing."""
    a = Setup(w4, "int8", 128, 4, 7, 16, 1, [3000, 900], seed=1)
    b = Setup(w4, "int8", 128, 4, 7, 16, 2, [2500, 17, 1300], seed=2)
    want_a = a.cache.attend(a.gq, a.glens, a.table)
    # b over a's cache object: its pool and table, a's workspaces
    b.cache.attend(b.gq, b.glens, b.table)
    want_b = b.cache.attend(b.gq, b.glens, b.table, workspace=b.cache.new_workspace())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.cache.attend(a.gq, a.glens, a.table)
        of_side = a.cache.workspace
    assert of_side is not None and of_side.data_ptr() != a.cache.workspace.data_ptr()
    a.cache.attend(a.gq, a.glens, a.table, stream=side)        # by argument: the same one
    with torch.cuda.stream(side):
        assert a.cache.workspace is of_side
    torch.cuda.synchronize()
    # a captured call leaves the eager ones' workspaces alone, and keeps none
    mine, kept = a.cache.workspace, a.cache.workspace.clone()
    out, lse = torch.empty_like(want_a[0]), torch.empty_like(want_a[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.cache.attend(a.gq, a.glens, a.table, out=out, lse=lse)
        a.cache.attend(a.gq, a.glens, a.table, out=out, lse=lse)
    assert a.cache.workspace is mine
    torch.cuda.synchronize()
    mine.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want_a[0]) and torch.equal(lse, want_a[1])
    assert (mine == 0).all()
    mine.copy_(kept)
    # the first call of a cache under capture
    new = w4.PagedCache(a.cache.pool, a.cache.format, 4, 128)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        new.attend(a.gq, a.glens, a.table, out=out, lse=lse)
    assert new.workspace is None
    # side by side
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        got.append(a.cache.attend(a.gq, a.glens, a.table))
        graph.replay()
        got.append(a.cache.attend(a.gq, a.glens, a.table, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want_a[0]) and torch.equal(x, want_a[1]) for o, x in got)
    assert torch.equal(out, want_a[0])
    got = b.cache.attend(b.gq, b.glens, b.table)
    assert torch.equal(got[0], want_b[0]) and torch.equal(got[1], want_b[1])


def test_infinite_values_of_visible_keys_stay_infinite(w4):  # noqa: F811
    """bf16: an infinite value gives an infinite result of its sign in its
    column for every row that sees it (however round its probability is), and
    changes no other column."""
    for M, n in ((1, 50), (4, 37), (1, 1)):
        s = Setup(w4, "bf16", 64, 1, 2, 16, M, [n], seed=n)
        want, want_lse = s.cache.attend(s.gq, s.glens, s.table)
        for bad in (float("inf"), float("-inf")):
            v = s.values[0].copy()
            v[0, 0, 5] = v[n // 2, 0, 5] = bad                 # all rows see these keys
            s.cache.append(to_gpu(s.keys[0]), to_gpu(v), i32(np.arange(n)), s.table)
            got, lse = s.cache.attend(s.gq, s.glens, s.table)
            assert (got[..., 5] == bad).all()
            keep = torch.arange(64, device="cuda") != 5
            assert torch.equal(got[..., keep], want[..., keep]) and torch.equal(lse, want_lse)
    # equal scores: every probability is a power of two
    s.gq.zero_()
    got, _ = s.cache.attend(s.gq, s.glens, s.table)
    assert (got[..., 5] == float("-inf")).all()


@pytest.mark.parametrize("D,H,group,M", [(128, 4, 7, 1), (64, 2, 7, 3), (128, 2, 4, 8)])
def test_probabilities_beside_bf16_values_keep_16_bits(w4, D, H, group, M):  # noqa: F811
    """The fp32 result of a bf16 cache: probabilities within 2^-15 of
    themselves (their two parts), scores as in kv_testutil."""
    lens = [900, 33, 8, 400]
    s = Setup(w4, "bf16", D, H, group, 16, M, lens, seed=D + M)
    out = torch.empty(s.gq.shape, device="cuda")
    w4.paged_attn_f32(s.cache, s.gq, out, s.glens, s.table, s.cache.new_workspace())
    ref, _, mag = kv.attention(s.q, s.keys, s.values, lens, M, D ** -0.5, 0)
    dS = kv.score_error("bf16", s.q, s.keys, s.scales, lens, D ** -0.5)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= (2.0 ** -15 + 4 * dS + (max(lens) + 64) * 2.0 ** -23) * mag + 1e-30).all()
    # the scores' errors have both signs and are far from their bound
    assert np.linalg.norm(err) <= (2.0 ** -15 + 2.0 ** -15) * np.linalg.norm(mag)


def test_a_workspace_of_the_callers_can_be_set(w4):  # noqa: F811
    s = Setup(w4, "int4", 64, 2, 3, 16, 1, [700, 40], seed=1)
    want = s.cache.attend(s.gq, s.glens, s.table)
    mine = s.cache.new_workspace().fill_(0)
    s.cache.workspace = mine
    got = s.cache.attend(s.gq, s.glens, s.table)
    assert s.cache.workspace is mine and bool((mine != 0).any())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    s.cache.workspace = None
    got = s.cache.attend(s.gq, s.glens, s.table)
    assert s.cache.workspace is not mine and torch.equal(got[0], want[0])
