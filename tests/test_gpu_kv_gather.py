"""w4_kv_gather, byte by byte: every format, head layout and page size, lists that
end inside a record, repeat, run backwards, leave places out or point nowhere, all
that is to stay as it was, weights beside the tokens, streams, graphs, offsets past 32
bits, refusals; and the whole way of an eviction: attention, weights, selection,
moving, and the attention over what is left."""
import numpy as np
import pytest

from tests import kv_testutil as kv
from tests.test_gpu_paged_attn import Setup, i32, to_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

MARK = 7.0


@pytest.fixture(scope="module")
def w4():
    from int4_weight_only_w4_gb300 import w4 as mod
    return mod


class Host:
    """Pool bytes on the host, [pages, heads, records, bytes], and tokens' bytes in them."""

    def __init__(self, pool, fmt, D, H, P):
        self.fmt, self.D, self.P = fmt, D, P
        self.bytes = pool.cpu().numpy().reshape(-1, H, P // 16, kv.record_bytes(fmt, D)).copy()

    def move(self, head, src, dst):
        """The token at (page, place) src of a head, as it is held, to dst."""
        a = self.bytes[src[0], head, src[1] // 16].copy()
        b = self.bytes[dst[0], head, dst[1] // 16]
        r0, r1 = src[1] % 16, dst[1] % 16
        for which in (0, 1):
            p0, p1 = (kv.places(self.fmt, self.D)[which][r] for r in (r0, r1))
            if self.fmt == "bf16":
                for y in (0, 1):
                    b[p1[:, 0] + y] = a[p0[:, 0] + y]
                continue
            if self.fmt == "int8":
                b[p1[:, 0]] = a[p0[:, 0]]
            else:
                code = (a[p0[:, 0]] >> (4 * p0[:, 1]).astype(np.uint8)) & 15
                for n in (0, 1):
                    m = p1[:, 1] == n
                    keep = 0xF0 if n == 0 else 0x0F
                    b[p1[m, 0]] = (b[p1[m, 0]] & keep) | (code[m] << (4 * n)).astype(np.uint8)
            o = len(a) - 128 + 64 * which
            b[o + 4 * r1:o + 4 * r1 + 4] = a[o + 4 * r0:o + 4 * r0 + 4]


class Moving:
    """A cache with tokens in some pages (Setup) and as many free ones as `most` places
    of every sequence take, filled with random bytes."""

    def __init__(self, w4, fmt, D, H, P, lens, most, group=1, M=1, seed=0):
        s = self.s = Setup(w4, fmt, D, H, group, P, M, lens, seed=seed)
        self.w4, self.fmt, self.D, self.H, self.P, self.lens, self.most = \
            w4, fmt, D, H, P, lens, most
        B, width = len(lens), -(-most // P)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        per_page = s.cache.pool.numel() // s.cache.pages
        free = torch.randint(0, 256, (B * width * per_page,), generator=gen, device="cuda",
                             dtype=torch.uint8)
        self.cache = w4.PagedCache(torch.cat([s.cache.pool, free]), kv.FMT[fmt], H, D, P)
        order = torch.randperm(B * width, generator=gen, device="cuda") + s.cache.pages
        self.to = order.view(B, width).to(torch.int32)
        self.rng = np.random.default_rng(seed)

    def lists(self, counts):
        """Random ascending indices of every head."""
        index = np.full((len(self.lens), self.H, self.most), -5)
        for b, c in enumerate(counts):
            for h in range(self.H):
                index[b, h, :c] = np.sort(self.rng.permutation(self.lens[b])[:c])
        return index

    def check(self, index, counts, weights=True, **kw):
        """Call, and compare the whole pool and all weights."""
        host = Host(self.cache.pool, self.fmt, self.D, self.H, self.P)
        table, to = self.s.table.cpu().numpy(), self.to.cpu().numpy()
        columns = max(max(self.lens), 1)
        w = self.rng.random((len(self.lens), self.H, columns)).astype(np.float32)
        want = np.full((len(self.lens), self.H, self.most), MARK, np.float32)
        for b, c in enumerate(counts):
            for h in range(self.H):
                for i in range(min(max(c, 0), self.most)):
                    j = index[b][h][i]
                    if 0 <= j < self.lens[b]:
                        host.move(h, (table[b, j // self.P], j % self.P),
                                  (to[b, i // self.P], i % self.P))
                        want[b, h, i] = w[b, h, j]
        out = torch.full((*want.shape[:2], self.most + self.most % 3), MARK, device="cuda")
        pair = dict(weights=torch.from_numpy(w).cuda(), weights_out=out) if weights else {}
        self.cache.gather(self.s.table, self.s.glens, i32(index), i32(counts), self.to, **pair,
                          **kw)
        torch.cuda.synchronize()
        got = self.cache.pool.cpu().numpy().reshape(host.bytes.shape)
        assert np.array_equal(got, host.bytes)
        if weights:
            got = out.cpu().numpy()
            assert np.array_equal(got[..., :self.most], want) and (got[..., self.most:] == MARK).all()


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257]


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D,H,P", [(128, 4, 16), (64, 2, 32), (128, 1, 64), (64, 3, 16),
                                   (128, 2, 48), (64, 1, 128)])
def test_formats(w4, fmt, D, H, P):
    for most in (1, 16, 37):
        m = Moving(w4, fmt, D, H, P, LENS, most, seed=D + most)
        m.check(m.lists([min(n, most) for n in LENS]), [min(n, most) for n in LENS])
        m.check(m.lists([min(n, most) // 2 for n in LENS]), [min(n, most) // 2 for n in LENS],
                weights=False)
        m.cache.check()


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D", [64, 128])
def test_any_order(w4, fmt, D):
    """Backwards, the same token again and again, places left out."""
    m = Moving(w4, fmt, D, 2, 32, [90, 200], 50, seed=D)
    back = np.arange(50)[::-1] + 30
    m.check(np.tile(back, (2, 2, 1)), [50, 45])
    m.check(np.full((2, 2, 50), 17), [50, 33])
    some = np.tile(np.arange(50), (2, 2, 1))
    some[:, 0, ::3] = -1
    some[1, 1, :16], some[0, 1, 16:32] = -(2 ** 31), -7
    m.check(some, [50, 50])
    m.check(m.rng.integers(0, 90, (2, 2, 50)), [49, 17])
    m.cache.check()


def test_what_points_nowhere(w4):
    m = Moving(w4, "int4", 64, 2, 16, [40, 70], 20, seed=3)
    index = m.lists([20, 20])
    index[0, 0, 3], index[1, 1, 7], index[0, 1, 0] = 40, 2 ** 31 - 1, 41
    m.check(index, [20, 20])
    assert m.cache.error.item() == w4.KV_ERR_POSITION
    m.cache.error.zero_()
    m.check(m.lists([20, 20]), [21, -4])
    assert m.cache.error.item() == w4.KV_ERR_LENGTH
    m.cache.error.zero_()
    # pages that are not in the pool, on either side
    before, index = m.cache.pool.clone(), i32(m.lists([20, 20]))
    bad = torch.full_like(m.to, 10 ** 7)
    m.cache.gather(m.s.table, m.s.glens, index, i32([20, 20]), bad)
    torch.cuda.synchronize()
    assert m.cache.error.item() == w4.KV_ERR_PAGE and torch.equal(m.cache.pool, before)
    m.cache.error.zero_()
    m.cache.gather(torch.full_like(m.s.table, -1), m.s.glens, index, i32([20, 20]), m.to)
    torch.cuda.synchronize()
    assert m.cache.error.item() == w4.KV_ERR_PAGE and torch.equal(m.cache.pool, before)
    m.cache.error.zero_()
    # weights for some of the tokens only: the others are not there
    w = torch.ones(2, 2, 10, device="cuda")
    out = torch.full((2, 2, 20), MARK, device="cuda")
    ahead = np.tile(np.arange(20), (2, 2, 1))
    m.cache.gather(m.s.table, m.s.glens, i32(ahead), i32([20, 20]), m.to, w, out)
    torch.cuda.synchronize()
    assert m.cache.error.item() == w4.KV_ERR_POSITION
    assert (out[..., :10] == 1).all() and (out[..., 10:] == MARK).all()


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_many_sequences(w4, fmt):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 40, 300).tolist()
    m = Moving(w4, fmt, 64, 1, 16, lens, 20, seed=2)
    counts = [min(n, 20) for n in lens]
    m.check(m.lists(counts), counts)
    m.cache.check()


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_an_eviction(w4, fmt):
    """Attention, its weights, the heaviest tokens and the newest ones, moved; then the
    attention over what is left is that over those keys, and goes on from there."""
    P, M, H, D, lens, count = 16, 1, 2, 64, [300, 20, 0, 150], 48
    m = Moving(w4, fmt, D, H, P, lens, count + 16, group=3, seed=6)
    s, c, B = m.s, m.cache, len(lens)
    s.cache = c
    _, lse = c.attend(s.gq, s.glens, s.table)
    weights = c.attn_weights(s.gq, lse, s.glens, s.table, columns=320)
    index = torch.full((B, H, count), -1, device="cuda", dtype=torch.int32)
    counts = torch.zeros(B, device="cuda", dtype=torch.int32)
    w4.select(weights, s.glens, index, counts, first=2, last=10)
    kept = c.gather(s.table, s.glens, index, counts, m.to, weights)
    c.check()
    chosen, n = index.cpu().numpy(), counts.cpu().numpy()
    assert (n == [48, 20, 0, 48]).all()
    host = weights.cpu().numpy()
    out, lse = c.attend(s.gq, counts, m.to)
    for b in range(B):
        for h in range(H):
            pick = chosen[b, h, :n[b]]
            assert np.array_equal(kept[b, h, :n[b]].cpu().numpy(), host[b, h, pick])
            if not n[b]:
                continue
            ref = kv.attention(s.q[b:b + 1, 3 * h:3 * h + 3], [s.keys[b][pick][:, h:h + 1]],
                               [s.values[b][pick][:, h:h + 1]], [n[b]], 1, D ** -0.5, 0)
            dS = kv.score_error(fmt, s.q, s.keys, s.scales, lens, D ** -0.5)
            kv.check_attention(out[b:b + 1, 3 * h:3 * h + 3].float().cpu().numpy(),
                               lse[b:b + 1, 3 * h:3 * h + 3].cpu().numpy(), *ref, fmt, dS, 48, True)
    # the next token goes behind the kept ones, whose weights go on from what they were
    k = to_gpu(m.rng.standard_normal((B, H, D)).astype(np.float32))
    c.append(k, k, counts, m.to)
    lens, before = counts + 1, kept.clone()
    c.attn_weights(s.gq, c.attend(s.gq, lens, m.to)[1], lens, m.to, before=kept, weights=kept)
    added = (kept - before).double().sum(-1)
    assert kept.shape == weights.shape and ((added - 3).abs() <= 1e-4).all()   # one a row
    for b, n in enumerate(lens.tolist()):
        assert (kept[b, :, :n] >= before[b, :, :n]).all() and (kept[b, :, n:] == 0).all()
    c.check()


def test_stream_graph_and_repeats(w4):
    m = Moving(w4, "int8", 128, 2, 16, [100, 1, 700], 60, seed=3)
    counts = [60, 1, 60]
    index = m.lists(counts)
    m.check(index, counts)
    want = m.cache.pool.clone()
    gi, gc = i32(index), i32(counts)
    free = slice(m.s.cache.pool.numel(), None)
    side = torch.cuda.Stream()
    for _ in range(3):
        m.cache.pool[free] = want[free] ^ 255
        side.wait_stream(torch.cuda.current_stream())
        m.cache.gather(m.s.table, m.s.glens, gi, gc, m.to, stream=side)
        side.synchronize()
        kept = m.cache.pool.clone()
        m.cache.gather(m.s.table, m.s.glens, gi, gc, m.to)
        assert torch.equal(m.cache.pool, kept)
    k0, v0 = m.cache.read(torch.arange(60, device="cuda", dtype=torch.int32), m.to,
                          seq_ids=torch.zeros(60, device="cuda", dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.cache.gather(m.s.table, m.s.glens, gi, gc, m.to)
    m.cache.pool[free] = want[free]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(m.cache.pool, want)


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
    old, new = i32([[pages - 1, 5, pages // 2 + 3]]), i32([[pages - 2, pages // 2, 9]])
    for a, b in zip(s.table[0, :3].tolist(), old[0].tolist()):
        cache.pool.view(-1, per_page)[b] = s.cache.pool.view(-1, per_page)[a]
    index = i32(np.tile(np.arange(32, -1, -1), (1, H, 1)))
    cache.gather(old, s.glens, index, s.glens, new)
    pos = torch.arange(33, device="cuda", dtype=torch.int32)
    for a, b in zip(cache.read(pos, new), cache.read(32 - pos, old)):
        assert torch.equal(a, b)
    cache.check()


def test_refusals(w4):
    m = Moving(w4, "bf16", 64, 2, 16, [40, 70], 20, seed=3)
    index, counts = i32(m.lists([20, 20])), i32([20, 20])
    w, out = torch.zeros(2, 2, 70, device="cuda"), torch.zeros(2, 2, 20, device="cuda")
    args = dict(table=m.s.table, lens=m.s.glens, index=index, counts=counts, to=m.to, weights=w,
                weights_out=out)
    call = lambda **kw: w4.kv_gather(m.cache, **dict(args, **kw))  # noqa: E731
    call()
    for kw in (dict(index=index[:1]), dict(index=index.long()), dict(counts=counts[:1]),
               dict(lens=m.s.glens[:1]), dict(weights=None), dict(weights_out=None),
               dict(weights=w[:1]), dict(weights_out=out[:1]),
               dict(weights=w.double()), dict(index=index.cpu()), dict(to=m.to.long())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(to=m.to[:1]), dict(to=m.s.table),
               dict(weights_out=out[..., :10].contiguous())):
        with pytest.raises(w4.W4Error) as e:
            call(**kw)
        assert e.value.status == w4.Status.INVALID_ARG
