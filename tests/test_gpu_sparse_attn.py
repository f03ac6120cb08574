"""w4_sparse_attn against fp64 over the listed blocks of what the cache holds:
formats, head layouts, page sizes, 1-8 new tokens, lists of every length (none,
all, different ones a head), blocks that a row does not reach, entries that are
left out, what lies past the length (NaN), strides, streams, graphs, and the whole
way of a step: bounds, scores, selection, attention.  Tolerances: kv_testutil."""
import numpy as np
import pytest

from tests import kv_testutil as kv
from tests.test_gpu_paged_attn import Setup, i32, to_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500]


@pytest.fixture(scope="module")
def w4():
    from int4_weight_only_w4_gb300 import w4 as mod
    return mod


def lists(rng, lens, H, P, most):
    """Random ascending lists of up to `most` blocks, -1 past their ends, and counts."""
    blocks = np.full((len(lens), H, most), -1)
    counts = np.zeros(len(lens), int)
    for b, n in enumerate(lens):
        there = -(-max(n, 0) // P)
        counts[b] = c = min(there, int(rng.integers(0, most + 1)))
        for h in range(H):
            blocks[b, h, :c] = np.sort(rng.permutation(there)[:c])
    return blocks, counts


def reference(s, P, chosen, scale):
    """chosen[b][h]: the blocks that count.  out, lse, A = sum p |v| as kv.attention."""
    T, HQ, D = s.q.shape
    H, M = s.cache.kv_heads, s.M
    G = HQ // H
    out, mag, lse = np.zeros((T, HQ, D)), np.zeros((T, HQ, D)), np.full((T, HQ), -np.inf)
    for b, n in enumerate(s.lens):
        for h in range(H):
            j = np.array([x for k in chosen[b][h] for x in range(k * P, min(n, k * P + P))], int)
            for i in range(M):
                seen = j[j <= n - M + i]
                if not len(seen):
                    continue
                k = s.keys[b][seen, h].astype(np.float64)
                v = s.values[b][seen, h].astype(np.float64)
                t, heads = b * M + i, slice(h * G, (h + 1) * G)
                x = s.q[t, heads].astype(np.float64) @ k.T * scale
                e = np.exp(x - x.max(-1, keepdims=True))
                total = e.sum(-1, keepdims=True)
                out[t, heads], mag[t, heads] = e / total @ v, e / total @ np.abs(v)
                lse[t, heads] = (x.max(-1, keepdims=True) + np.log(total))[:, 0]
    return out, lse, mag


def check(s, got, lse, P, chosen, scale=None, bf16_out=True, what=""):
    D = s.q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    dS = kv.score_error(s.fmt, s.q, s.keys, s.scales, s.lens, scale)
    kv.check_attention(got.float().cpu().numpy(), lse.cpu().numpy(), *reference(s, P, chosen, scale),
                       s.fmt, dS, max(max(s.lens), 1), bf16_out, what)


def taken(blocks, counts):
    return [[row[:c] for row in seq] for seq, c in zip(blocks, counts)]


def run_both(w4, s, P, blocks, counts, scale=None, chosen=None):
    chosen = taken(blocks, counts) if chosen is None else chosen
    gb, gc = i32(blocks), i32(counts)
    got, lse = s.cache.attend_blocks(s.gq, s.glens, s.table, gb, gc, scale=scale)
    check(s, got, lse, P, chosen, scale, what="bf16")
    out, lse2 = torch.full(s.gq.shape, 5.0, device="cuda"), torch.empty_like(lse)
    w4.sparse_attn_f32(s.cache, s.gq, out, s.glens, s.table, gb, gc, s.cache.workspace, scale, lse2)
    check(s, out, lse2, P, chosen, scale, bf16_out=False, what="fp32")
    assert torch.equal(out.to(torch.bfloat16), got) and torch.equal(lse, lse2)
    return got, lse


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D,H,group,P", [(128, 4, 7, 16), (64, 2, 7, 32), (128, 1, 1, 64),
                                         (64, 3, 5, 16), (128, 2, 8, 48), (64, 1, 12, 16),
                                         (128, 1, 33, 16)])
@pytest.mark.parametrize("M", [1, 3, 8])
def test_formats_and_heads(w4, fmt, D, H, group, P, M):
    lens = LENS[M % 2::2]
    s = Setup(w4, fmt, D, H, group, P, M, lens, seed=D + H + group + M)
    for most in (1, 5, 32):
        run_both(w4, s, P, *lists(np.random.default_rng(most), lens, H, P, most))
    s.cache.check()


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("P,M", [(16, 1), (64, 5)])
def test_all_blocks_are_the_whole_attention(w4, fmt, P, M):
    lens = [0, 1, 700, 33, 64, 1500]
    s = Setup(w4, fmt, 64, 2, 3, P, M, lens, seed=M)
    most = -(-1500 // P) + 2
    blocks = np.tile(np.arange(most), (len(lens), 2, 1))
    counts = [-(-n // P) for n in lens]
    got, lse = run_both(w4, s, P, blocks, counts)
    want, want_lse = s.cache.attend(s.gq, s.glens, s.table)
    s.check(got, lse)
    assert (lse == want_lse).float().mean() > 0.5        # mostly the same sums


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_long_lists_are_split(w4, fmt):
    """Lists that many blocks of the device share, next to short ones."""
    rng = np.random.default_rng(4)
    lens, P = [9000, 40, 6001, 0], 32
    s = Setup(w4, fmt, 64, 2, 7, P, 2, lens, seed=5)
    blocks, _ = lists(rng, lens, 2, P, 200)
    counts = np.array([200, 1, 150, 0])
    for b in range(4):
        for h in range(2):
            blocks[b, h, :counts[b]] = np.sort(rng.permutation(-(-lens[b] // P))[:counts[b]])
    run_both(w4, s, P, blocks, counts)
    s.cache.check()


def test_rows_that_see_nothing(w4):
    """The only listed block begins after the first new tokens, or there is none."""
    M, P = 8, 16
    for n in (20, 3, 33):
        s = Setup(w4, "bf16", 64, 2, 2, P, M, [n, n], seed=n)
        last = -(-n // P) - 1
        blocks = np.array([[[last], [0]], [[0], [0]]])
        got, lse = run_both(w4, s, P, blocks, [1, 0])
        assert (got[M:] == 0).all() and torch.isneginf(lse[M:]).all()
        rows = n - M + np.arange(M) < max(last * P, 0)
        assert (torch.isneginf(lse[:M, :2]).all(-1).cpu().numpy() ==
                (rows | (n - M + np.arange(M) < 0))).all()


def test_entries_that_are_left_out(w4):
    P, n = 16, 100                                        # blocks 0 .. 6
    s = Setup(w4, "int8", 64, 1, 2, P, 1, [n], seed=2)
    for row, left in (([3, 3], [3]), ([5, 2], [5]), ([-1, 4], [4]), ([0, 7], [0]),
                      ([1, 10 ** 9], [1]), ([-2 ** 31, 2], [2]), ([6, 6], [6]),
                      ([0, 2 ** 31 - 1], [0])):
        run_both(w4, s, P, [[row]], [2], chosen=[[left]])
        torch.cuda.synchronize()
        assert s.cache.error.item() == w4.KV_ERR_BLOCK
        s.cache.error.zero_()
    # counts outside the list's room
    run_both(w4, s, P, [[[1, 4]]], [7], chosen=[[[1, 4]]])
    run_both(w4, s, P, [[[1, 4]]], [-3], chosen=[[[]]])
    s.cache.check()
    table = s.table.clone()
    table[0, 4] = 10 ** 6
    got, lse = s.cache.attend_blocks(s.gq, s.glens, table, i32([[[1, 4]]]), i32([2]))
    torch.cuda.synchronize()
    assert s.cache.error.item() == w4.KV_ERR_PAGE
    s.cache.error.zero_()
    check(s, got, lse, P, [[[1]]])
    s.cache.attend_blocks(s.gq, s.glens, s.table[:, :3].contiguous(), i32([[[1, 2]]]), i32([2]))
    torch.cuda.synchronize()
    assert s.cache.error.item() == w4.KV_ERR_LENGTH
    s.cache.error.zero_()


def test_what_is_not_listed_is_not_looked_at(w4):
    """NaN and infinity in other blocks, and in keys and values past a row's position,
    reach nothing."""
    M, n, P = 4, 90, 32
    s = Setup(w4, "bf16", 64, 1, 2, P, M, [n], seed=5)
    blocks, counts = i32([[[0, 2]]]), i32([2])
    want, want_lse = s.cache.attend_blocks(s.gq, s.glens, s.table, blocks, counts)
    for bad in (float("inf"), float("-inf"), float("nan")):
        k, v = s.keys[0].copy(), s.values[0].copy()
        k[32:64], v[32:64] = bad, bad
        k[n - 1, 0, 3], v[n - 2, 0, 5], v[n - 1] = bad, bad, bad
        s.cache.append(to_gpu(k), to_gpu(v), i32(np.arange(n)), s.table)
        got, lse = s.cache.attend_blocks(s.gq, s.glens, s.table, blocks, counts)
        assert torch.equal(got[:M - 2], want[:M - 2]) and torch.equal(lse[:M - 1], want_lse[:M - 1])
        keep = torch.arange(64, device="cuda") != 5
        assert torch.equal(got[M - 2][:, keep], want[M - 2][:, keep])
        assert not torch.isfinite(got[M - 2][:, 5].float()).any()


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_a_step(w4, fmt):
    """Bounds, scores, selection and attention one after another, from the lengths on
    the device alone, also captured."""
    P, M, count, lens = 32, 1, 6, [1000, 0, 150, 33, 800]
    s = Setup(w4, fmt, 128, 2, 4, P, M, lens, seed=3)
    B, width = s.table.shape
    c, bounds = s.cache, s.cache.new_bounds()
    index = torch.zeros(B, 2, count, device="cuda", dtype=torch.int32)
    counts = torch.zeros(B, device="cuda", dtype=torch.int32)
    scores = torch.zeros(B, 2, width, device="cuda")
    out, lse = torch.empty_like(s.gq), torch.empty(s.gq.shape[:2], device="cuda")
    c.key_bounds(bounds, s.glens, s.table, tokens=1000)

    def step():
        c.key_bounds(bounds, s.glens, s.table)
        c.block_scores(bounds, s.gq, s.glens, s.table, scores=scores)
        w4.select(scores, s.glens, index, counts, unit=P, first=1, last=1)
        c.attend_blocks(s.gq, s.glens, s.table, index, counts, out=out, lse=lse)

    step()
    c.check()
    got, n = index.cpu().numpy(), counts.cpu().numpy()
    assert (n == [6, 0, 5, 2, 6]).all()
    check(s, out, lse, P, taken(got, n))
    # a score is a bound of q . k in its block (up to its sum's rounding), and no block
    # that is left out has a larger one than a chosen one that did not have to be
    top = scores.cpu().numpy()
    for b, length in enumerate(lens):
        for h in range(2):
            k = kv.bf16(s.keys[b][:, h]).astype(np.float64)
            q = s.q[b, 4 * h:4 * h + 4].astype(np.float64)
            there = -(-length // P)
            for i in range(there):
                part = k[i * P:(i + 1) * P]
                slack = 2.0 ** -14 * np.abs(q).sum(-1).max() * np.abs(part).max()
                assert (q @ part.T).max() <= top[b, h, i] + slack
            chosen = set(got[b, h, :n[b]].tolist())
            free = [top[b, h, i] for i in chosen - {0, there - 1}]
            left = [top[b, h, i] for i in set(range(there)) - chosen]
            assert not free or not left or min(free) >= max(left)
    want, want_lse = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (out, lse, scores):
            t.fill_(7.0)
        index.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_strides_stream_graph_and_repeats(w4):
    lens, P = [100, 1, 700, 0], 16
    s = Setup(w4, "int8", 128, 2, 7, P, 3, lens, seed=3)
    blocks, counts = lists(np.random.default_rng(8), lens, 2, P, 20)
    want, want_lse = run_both(w4, s, P, blocks, counts)
    gb, gc = i32(blocks), i32(counts)
    T, HQ, D = s.q.shape
    rows = torch.zeros(T, HQ + 4, D, device="cuda", dtype=torch.bfloat16)
    rows[:, 1:HQ + 1] = s.gq
    wide = torch.full((HQ, T, D), 3.0, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    got, _ = s.cache.attend_blocks(rows[:, 1:HQ + 1], s.glens, s.table, gb, gc, out=wide)
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        again, lse = s.cache.attend_blocks(s.gq, s.glens, s.table, gb, gc)
        other, _ = s.cache.attend_blocks(s.gq, s.glens, s.table, gb, gc, stream=side)
        assert torch.equal(again, want) and torch.equal(lse, want_lse)
    side.synchronize()
    assert torch.equal(other, want)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.attend_blocks(s.gq, s.glens, s.table, gb, gc, out=out, lse=lse)
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


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
    run_both(w4, s, P, [[[0, 2], [1, 2], [0, 1], [0, 2]]], [2])
    cache.check()


def test_refusals(w4):
    s = Setup(w4, "int4", 64, 2, 2, 16, 1, [5, 6], seed=1)
    blocks, counts = torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda"), i32([1, 1])
    ws = s.cache.new_workspace()
    call = s.cache.attend_blocks
    call(s.gq, s.glens, s.table, blocks, counts)
    for b, c in ((blocks[:1], counts), (blocks[:, :1], counts), (blocks.long(), counts),
                 (blocks[0], counts), (blocks, counts[:1]), (blocks.cpu(), counts),
                 (blocks.expand(2, 2, 3), counts)):
        with pytest.raises(ValueError):
            call(s.gq, s.glens, s.table, b, c)
    with pytest.raises(w4.W4Error) as e:
        call(s.gq, s.glens, s.table, blocks[..., :0], counts)
    assert e.value.status == w4.Status.INVALID_ARG
    with pytest.raises(w4.W4Error):
        call(s.gq, s.glens, s.table, blocks, counts, workspace=ws[:256])
    with pytest.raises(w4.W4Error):
        call(s.gq, s.glens, s.table, blocks, counts, scale=float("nan"))
