"""w4_paged_attn against fp64 over the values that the cache holds: formats,
head layouts, 1-8 new tokens, lengths of zero, one and around every tile and
page border, windows, rows that see nothing, what lies past the length (NaN),
scales, strides, other streams, graphs, offsets past 32 bits, repeatability."""
import numpy as np
import pytest

from tests import kv_testutil as kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def w4():
    from int4_weight_only_w4_gb300 import w4 as mod
    return mod


def to_gpu(x):
    return torch.from_numpy(kv.bf16_bits(x).view(np.int16)).cuda().view(torch.bfloat16)


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


class Setup:
    """A cache filled on the host; everything outside the sequences' tokens is
    0xFF: NaN for bf16, NaN scales and zero points of 65535 otherwise."""

    def __init__(self, w4, fmt, D, H, group, P, M, lens, seed=0, spread=1.0, spare=2):
        rng = np.random.default_rng(seed)
        self.fmt, self.M, self.lens = fmt, M, list(lens)
        B, HQ = len(lens), H * group
        width = max(1, -(-max(lens) // P)) + 1
        table = rng.permutation(B * width + spare)[:B * width].reshape(B, width).astype(np.int32)
        host = kv.Pool(fmt, D, H, P, B * width + spare)
        self.keys, self.values, self.scales = [], [], []
        chan = np.where(rng.random((H, D)) < 1 / 16, 4, 1).astype(np.float32)
        for b, n in enumerate(lens):
            k = kv.bf16(rng.standard_normal((n, H, D)).astype(np.float32) * chan * spread)
            v = kv.bf16(rng.standard_normal((n, H, D)).astype(np.float32) + 0.25)
            for t in range(n):
                host.write(table[b, t // P], t % P, k[t], v[t])
            self.keys.append(kv.held(k, fmt) if n else k)
            self.values.append(kv.held(v, fmt) if n else v)
            self.scales.append(kv.quantise(k, fmt)[1].astype(np.float32)
                               if fmt != "bf16" and n else np.zeros(1, np.float32))
            # pages past the length are not there
            table[b, -(-n // P):] = -1 if b % 2 else 10 ** 9
        self.q = kv.bf16(rng.standard_normal((B * M, HQ, D)).astype(np.float32))
        self.host, self.table = host, i32(table)
        self.cache = w4.PagedCache(torch.from_numpy(host.bytes).cuda().view(-1), kv.FMT[fmt], H, D,
                                   P)
        self.gq, self.glens = to_gpu(self.q), i32(lens)

    def check(self, got, lse, scale=None, window=0, bf16_out=True, what=""):
        D = self.q.shape[2]
        scale = D ** -0.5 if scale is None else scale
        ref = kv.attention(self.q, self.keys, self.values, self.lens, self.M, scale, window)
        dS = kv.score_error(self.fmt, self.q, self.keys, self.scales, self.lens, scale)
        kv.check_attention(got.float().cpu().numpy(), lse.cpu().numpy(), *ref, self.fmt, dS,
                           max(max(self.lens), 1), bf16_out, what)
        self.cache.check()


def run_both(w4, s, scale=None, window=0):
    got, lse = s.cache.attend(s.gq, s.glens, s.table, scale=scale, window=window)
    s.check(got, lse, scale, window, what="bf16")
    out = torch.full(s.gq.shape, 5.0, device="cuda")
    lse2 = torch.empty_like(lse)
    w4.paged_attn_f32(s.cache, s.gq, out, s.glens, s.table, s.cache.workspace, scale, window, lse2)
    s.check(out, lse2, scale, window, bf16_out=False, what="fp32")
    # bf16 is the fp32 result rounded once
    assert torch.equal(out.to(torch.bfloat16), got) and torch.equal(lse, lse2)
    return got, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500]


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D,H,group,P", [(128, 4, 7, 16), (64, 2, 7, 32), (128, 1, 1, 64),
                                         (64, 3, 5, 16), (128, 2, 8, 48), (64, 1, 12, 16),
                                         (128, 1, 33, 16)])
@pytest.mark.parametrize("M", [1, 3, 8])
def test_formats_and_heads(w4, fmt, D, H, group, P, M):
    run_both(w4, Setup(w4, fmt, D, H, group, P, M, LENS[M % 2::2], seed=D + H + group + M))


@pytest.mark.parametrize("M", range(1, 9))
def test_every_token_count(w4, M):
    run_both(w4, Setup(w4, "bf16", 128, 4, 7, 16, M, [M - 1, 40, 300], seed=M))
    run_both(w4, Setup(w4, "int4", 64, 2, 7, 16, M, [M, 41, 301], seed=M))


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("lens", [[0], [1], [5, 0], [0, 0, 0, 0], [16], [700], [3000], [1100, 7],
                                  [2, 1500, 0, 900, 16, 33, 1]])
def test_lengths(w4, fmt, lens):
    for M in (1, 5):
        run_both(w4, Setup(w4, fmt, 64, 2, 3, 16, M, lens, seed=len(lens) + M))


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 4000])
def test_windows(w4, fmt, window):
    s = Setup(w4, fmt, 128, 2, 4, 32, 4, [0, 1, 3, 16, 19, 100, 117, 333, 900], seed=window)
    run_both(w4, s, window=window)


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 1e-4])
def test_scales(w4, fmt, scale):
    """Also scores so far apart that one key takes everything."""
    s = Setup(w4, fmt, 128, 1, 7, 16, 2, [1, 70, 350], seed=9)
    run_both(w4, s, scale=scale)


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_many_sequences(w4, fmt):
    """More sequences than the schedule scans at once, most of them short."""
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 40, 700)
    lens[[3, 400, 699]] = [600, 0, 333]
    run_both(w4, Setup(w4, fmt, 64, 1, 4, 16, 1, lens.tolist(), seed=12))


def test_values_of_zero_and_infinite_draft_keys(w4):
    """All-zero values (scale 0) give zero; an infinite value that a row does
    not see does not reach it."""
    for fmt in kv.FMT:
        s = Setup(w4, fmt, 64, 1, 2, 16, 1, [37], seed=4)
        zero = torch.zeros(37, 1, 64, device="cuda", dtype=torch.bfloat16)
        s.cache.append(to_gpu(s.keys[0]), zero, i32(np.arange(37)), s.table)
        got, lse = s.cache.attend(s.gq, s.glens, s.table)
        assert (got == 0).all() and torch.isfinite(lse).all()
    M, n = 4, 50
    s = Setup(w4, "bf16", 64, 1, 2, 16, M, [n], seed=5)
    want, want_lse = s.cache.attend(s.gq, s.glens, s.table)
    for bad in (float("inf"), float("-inf"), float("nan")):
        k, v = s.keys[0].copy(), s.values[0].copy()
        k[n - 1, 0, 3], v[n - 2, 0, 5], v[n - 1] = bad, bad, bad
        s.cache.append(to_gpu(k), to_gpu(v), i32(np.arange(n)), s.table)
        got, lse = s.cache.attend(s.gq, s.glens, s.table)
        # the rows before the draft tokens n-2 and n-1 are as they were
        assert torch.equal(got[:M - 2], want[:M - 2]) and torch.equal(lse[:M - 1], want_lse[:M - 1])
        # row M-2 sees v[n-2]: only its column 5 is not finite
        keep = torch.arange(64, device="cuda") != 5
        assert torch.equal(got[M - 2][:, keep], want[M - 2][:, keep])
        assert not torch.isfinite(got[M - 2][:, 5].float()).any()
    # the same in a key that the window leaves out, in the record where it starts
    s = Setup(w4, "bf16", 64, 1, 2, 16, 1, [n], seed=6)
    want, _ = s.cache.attend(s.gq, s.glens, s.table, window=10)
    k, v = s.keys[0].copy(), s.values[0].copy()
    k[:n - 10], v[:n - 10] = np.nan, np.inf
    s.cache.append(to_gpu(k), to_gpu(v), i32(np.arange(n)), s.table)
    got, _ = s.cache.attend(s.gq, s.glens, s.table, window=10)
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_long_sequences_are_split(w4, fmt):
    """Lengths that many blocks share, next to short ones: filled on the GPU
    and compared with fp64 on the GPU."""
    D, H, group, P, M = 128, 2, 7, 16, 2
    lens = [40000, 9, 17001]
    B, width = len(lens), 2500
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    cache = w4.PagedCache.make(B * width, kv.FMT[fmt], H, D, P)
    table = torch.randperm(B * width, generator=gen, device="cuda").view(B, width).to(torch.int32)
    q = torch.randn(B * M, H * group, D, generator=gen, device="cuda").to(torch.bfloat16)
    held = []
    for b, n in enumerate(lens):
        k = (2 * torch.randn(n, H, D, generator=gen, device="cuda")).to(torch.bfloat16)
        v = torch.randn(n, H, D, generator=gen, device="cuda").to(torch.bfloat16)
        pos = torch.arange(n, device="cuda", dtype=torch.int32)
        cache.append(k, v, pos, table, seq_ids=torch.full_like(pos, b))
        if fmt == "bf16":
            held.append((k.double(), v.double()))
        else:
            x = [kv.held(t.float().cpu().numpy(), fmt) for t in (k, v)]
            held.append(tuple(torch.from_numpy(t).cuda().double() for t in x))
    for window in (0, 12345):
        got, lse = cache.attend(q, i32(lens), table, window=window)
        cache.check()
        for b, n in enumerate(lens):
            k, v = held[b]
            for i in range(M):
                last = n - M + i
                first = max(0, last + 1 - window) if window else 0
                qq = q[b * M + i].double().view(H, group, D)
                x = torch.einsum("hgd,jhd->hgj", qq, k[first:last + 1]) / D ** 0.5
                p = torch.softmax(x, -1)
                ref = torch.einsum("hgj,jhd->hgd", p, v[first:last + 1]).reshape(-1, D)
                mag = torch.einsum("hgj,jhd->hgd", p, v[first:last + 1].abs()).reshape(-1, D)
                err = (got[b * M + i].double() - ref)
                u = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -10
                # the statistical form of kv_testutil's bound: errors of both
                # signs over many keys add up like their root mean square
                assert err.norm() <= u * (p.square().sum(-1).sqrt().max() * 4) * mag.norm() \
                    + 2.0 ** -8 * ref.norm() + 2.0 ** -12 * mag.norm(), (fmt, b, i)
                want = torch.logsumexp(x, -1).reshape(-1)
                assert (lse[b * M + i].double() - want).abs().max() <= 1e-4


def test_strides_stream_graph_and_repeats(w4):
    s = Setup(w4, "int8", 128, 2, 7, 16, 3, [100, 1, 700, 0], seed=3)
    want, want_lse = run_both(w4, s)
    T, HQ, D = s.q.shape
    rows = torch.zeros(T, HQ + 4, D, device="cuda", dtype=torch.bfloat16)
    rows[:, 1:HQ + 1] = s.gq
    wide = torch.full((HQ, T, D), 3.0, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    got, _ = s.cache.attend(rows[:, 1:HQ + 1], s.glens, s.table, out=wide)
    assert torch.equal(got, want)
    for _ in range(20):
        again, lse = s.cache.attend(s.gq, s.glens, s.table)
        assert torch.equal(again, want) and torch.equal(lse, want_lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again, _ = s.cache.attend(s.gq, s.glens, s.table, workspace=s.cache.new_workspace())
    side.synchronize()
    assert torch.equal(again, want)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.attend(s.gq, s.glens, s.table, out=out, lse=lse)
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # the lengths are read by the kernel: a replay sees new ones
    s.glens.copy_(i32([20, 5, 300, 1]))
    s.lens = [20, 5, 300, 1]
    s.keys = [k[:n] if len(k) >= n else k for k, n in zip(s.keys, s.lens)]
    graph.replay()
    torch.cuda.synchronize()
    for b, n in ((0, 20), (2, 300)):
        one = Setup.__new__(Setup)
        one.__dict__.update(s.__dict__)
        ref, ref_lse, mag = kv.attention(s.q[b * 3:b * 3 + 3], [s.keys[b]], [s.values[b][:n]], [n],
                                         3, 128 ** -0.5, 0)
        dS = kv.score_error("int8", s.q, [s.keys[b]], [s.scales[b]], [n], 128 ** -0.5)
        kv.check_attention(out[b * 3:b * 3 + 3].float().cpu().numpy(),
                           lse[b * 3:b * 3 + 3].cpu().numpy(), ref, ref_lse, mag, "int8", dS, n,
                           True)


def test_bad_pages_and_lengths_are_recorded(w4):
    s = Setup(w4, "bf16", 64, 2, 2, 16, 1, [40, 50], seed=8)
    table = s.table.clone()
    table[0, 1] = 1000
    got, lse = s.cache.attend(s.gq, s.glens, table)
    torch.cuda.synchronize()
    assert s.cache.error.item() == w4.KV_ERR_PAGE
    # sequence 0 goes on without the page's keys; sequence 1 is whole
    keep = np.r_[0:16, 32:40]
    ref = kv.attention(s.q, [s.keys[0][keep], s.keys[1]], [s.values[0][keep], s.values[1]],
                       [24, 50], 1, 64 ** -0.5, 0)
    dS = kv.score_error("bf16", s.q, s.keys, s.scales, s.lens, 64 ** -0.5)
    kv.check_attention(got.float().cpu().numpy(), lse.cpu().numpy(), *ref, "bf16", dS, 50, True)
    s.cache.error.zero_()
    short = s.table[:, :3].contiguous()                    # room for 48 tokens
    s.cache.attend(s.gq, i32([40, 50]), short)
    torch.cuda.synchronize()
    assert s.cache.error.item() == w4.KV_ERR_LENGTH
    s.cache.error.zero_()
    got, lse = s.cache.attend(s.gq, i32([-5, 50]), s.table)
    assert (got[0] == 0).all() and torch.isneginf(lse[0]).all()
    s.cache.check()


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
    src = s.cache.pool.view(-1, per_page)
    dst = cache.pool.view(-1, per_page)
    for a, b in zip(s.table[0, :3].tolist(), table[0].tolist()):
        dst[b] = src[a]
    s.cache, s.table = cache, table
    run_both(w4, s)


def test_refusals(w4):
    s = Setup(w4, "int4", 64, 2, 2, 16, 1, [5, 6], seed=1)
    ws = s.cache.new_workspace()

    def call(q=s.gq, out=None, lens=s.glens, table=s.table, ws=ws, **kw):
        out = torch.empty(q.shape, device="cuda", dtype=torch.bfloat16) if out is None else out
        w4.paged_attn(s.cache, q, out, lens, table, ws, **kw)

    def status(**kw):
        with pytest.raises(w4.W4Error) as e:
            call(**kw)
        return e.value.status

    call()
    with pytest.raises(ValueError):
        call(q=s.gq[:1])
    with pytest.raises(ValueError):
        call(q=s.gq.float())
    with pytest.raises(ValueError):
        call(lens=s.glens[:1])
    with pytest.raises(ValueError):
        call(out=torch.empty(2, 4, 64, device="cuda"))
    with pytest.raises(ValueError):
        call(lse=torch.empty(2, 3, device="cuda"))
    assert status(window=-1) == w4.Status.INVALID_ARG
    assert status(scale=float("nan")) == w4.Status.INVALID_ARG
    assert status(ws=ws[:256]) == w4.Status.INVALID_ARG
    assert status(ws=ws[1:]) == w4.Status.INVALID_ARG
    assert status(q=s.gq[:, :3]) == w4.Status.INVALID_ARG          # 3 heads over 2
    nine = torch.zeros(18, 4, 64, device="cuda", dtype=torch.bfloat16)
    assert status(q=nine) == w4.Status.UNSUPPORTED
    odd = torch.zeros(2 * 4 * 64 + 4, device="cuda", dtype=torch.bfloat16)[4:].view(2, 4, 64)
    assert status(q=odd) == w4.Status.INVALID_ARG
    assert status(out=odd) == w4.Status.INVALID_ARG


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("power", [-60, 60])
def test_queries_of_any_size(w4, fmt, power):
    """Queries times a power of two with the scale divided by it: the same
    bits (every step scales exactly)."""
    s = Setup(w4, fmt, 64, 2, 7, 16, 2, [70, 33], seed=11)
    want, want_lse = run_both(w4, s)
    got, lse = s.cache.attend(s.gq * 2.0 ** power, s.glens, s.table, scale=64 ** -0.5 * 2.0 ** -power)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_keys_of_zero(w4, fmt):
    """All scores are 0 whatever the queries are: the mean of the values."""
    s = Setup(w4, fmt, 128, 1, 4, 16, 1, [50], seed=12, spread=0.0)
    s.q = kv.bf16(np.full_like(s.q, 1e35))
    s.gq = to_gpu(s.q)
    got, lse = s.cache.attend(s.gq, s.glens, s.table)
    s.check(got, lse)
    want = s.values[0].astype(np.float64).mean(0)              # [1, 128]
    u = 2.0 ** -8
    assert (np.abs(got[0].double().cpu().numpy() - want)
            <= 2 * u * np.abs(s.values[0]).mean(0)).all()
