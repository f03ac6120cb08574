"""w4_kv_append and w4_kv_read: the pool's bytes after writing against the
layout restated on the host, bit for bit, for every format; tokens in pieces,
in any order, over page borders; padding, bad pages and positions; offsets
past 32 bits; values that are not finite."""
import numpy as np
import pytest

from tests import kv_testutil as kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def w4():
    from int4_weight_only_w4_gb300 import w4 as mod
    return mod


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def to_gpu(x):
    return torch.from_numpy(kv.bf16_bits(x).view(np.int16)).cuda().view(torch.bfloat16)


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


def rows(rng, T, H, D):
    """Keys with some wide channels, some all-positive and some zero rows."""
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    x *= np.where(rng.random((H, D)) < 1 / 16, 6, 1).astype(np.float32)
    if T > 3:
        x[1] = np.abs(x[1])
        x[2] = -np.abs(x[2])
        x[3, 0] = 0
    return kv.bf16(x)


CASES = [  # D, kv heads, q heads, page, tokens per sequence, first position
    (128, 4, 28, 16, [1], [0]), (64, 2, 14, 16, [8], [13]), (128, 1, 1, 32, [37], [5]),
    (64, 3, 15, 48, [16, 16], [16, 3]), (128, 2, 16, 64, [70, 70, 70], [0, 61, 128]),
    (64, 8, 8, 16, [1] * 9, list(range(9))), (128, 4, 28, 128, [160], [96])]


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D,H,HQ,P,M,first", CASES)
@pytest.mark.parametrize("layout", [None, 0, 1])
def test_append_and_read(w4, fmt, D, H, HQ, P, M, first, layout):
    rng = np.random.default_rng(D + H + P + M[0] + (layout or 5))
    B, T = len(M), sum(M)
    width = max(f + m for f, m in zip(first, M)) // P + 2
    table = rng.permutation(B * width + 3)[:B * width].reshape(B, width).astype(np.int32)
    host = kv.Pool(fmt, D, H, P, B * width + 3)
    cache = w4.PagedCache(torch.from_numpy(host.bytes.copy()).cuda().view(-1), kv.FMT[fmt], H, D, P)
    fused = rows(rng, T, HQ + 2 * H, D)
    q, k, v = fused[:, :HQ], fused[:, HQ:HQ + H], fused[:, HQ + H:]
    pos = np.concatenate([np.arange(f, f + m) for f, m in zip(first, M)]).astype(np.int32)
    seq = np.repeat(np.arange(B), M)
    g = to_gpu(fused)
    gq, gk, gv = g[:, :HQ], g[:, HQ:HQ + H], g[:, HQ + H:]
    rope, kr, qr = None, k, q
    if layout is not None:
        rot = D if layout == 0 else D // 2
        tab = rng.uniform(-1, 1, (400, rot // 2, 2)).astype(np.float32)
        rope = w4.RopeTable(torch.from_numpy(tab).cuda(), layout)
        kr, qr = (kv.rotate(x, pos, tab, layout) for x in (k, q))
    for t in range(T):
        host.write(table[seq[t], pos[t] // P], pos[t] % P, kr[t], v[t])
    gtab = i32(table)
    cache.append(gk, gv, i32(pos), gtab, q=gq, q_out=gq, rope=rope)
    k2, v2 = cache.read(i32(pos), gtab)
    torch.cuda.synchronize()
    cache.check()
    got = cache.pool.cpu().numpy().reshape(host.bytes.shape)
    assert np.array_equal(got, host.bytes)          # and nothing beside the tokens
    assert np.array_equal(bits(gq), kv.bf16_bits(qr))
    for t in range(T):
        hk, hv = host.read(table[seq[t], pos[t] // P], pos[t] % P)
        assert np.array_equal(bits(k2[t]), kv.bf16_bits(hk)), t
        assert np.array_equal(bits(v2[t]), kv.bf16_bits(hv)), t
    # the same tokens in another order with explicit sequences, one by one too
    order = rng.permutation(T)
    again = w4.PagedCache(torch.full_like(cache.pool, 255), kv.FMT[fmt], H, D, P)
    gk2, gv2 = to_gpu(k[order]), to_gpu(v[order])
    cut = T // 3
    for a, b in ((0, cut), (cut, T)):
        again.append(gk2[a:b], gv2[a:b], i32(pos[order[a:b]]), gtab, seq_ids=i32(seq[order[a:b]]),
                     rope=rope)
    assert torch.equal(again.pool, cache.pool)
    k3, v3 = again.read(i32(pos[order]), gtab, seq_ids=i32(seq[order]))
    assert np.array_equal(bits(k3), bits(k2)[order]) and np.array_equal(bits(v3), bits(v2)[order])


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_strided_heads(w4, fmt):
    """Head-major k and v, and outputs that are slices of wider rows."""
    rng = np.random.default_rng(0)
    T, H, D = 20, 3, 64
    k, v = rows(rng, T, H, D), rows(rng, T, H, D)
    cache = w4.PagedCache.make(4, kv.FMT[fmt], H, D)
    table, pos = i32([[2, 0, 3]]), i32(np.arange(7, 7 + T))
    hm = [to_gpu(x.transpose(1, 0, 2)).transpose(0, 1) for x in (k, v)]
    cache.append(hm[0], hm[1], pos, table)
    wide = torch.full((T, 2 * H + 1, D), 9.0, device="cuda", dtype=torch.bfloat16)
    cache.read(pos, table, k=wide[:, :H], v=wide[:, H:2 * H])
    assert np.array_equal(bits(wide[:, :H]), kv.bf16_bits(kv.held(k, fmt)))
    assert np.array_equal(bits(wide[:, H:2 * H]), kv.bf16_bits(kv.held(v, fmt)))
    assert (wide[:, 2 * H] == 9.0).all()
    only = torch.empty(T, H, D, device="cuda", dtype=torch.bfloat16)
    w4.kv_read(cache, None, only, pos, table)
    assert np.array_equal(bits(only), kv.bf16_bits(kv.held(v, fmt)))


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_what_is_left_out(w4, fmt):
    rng = np.random.default_rng(1)
    T, H, D, P = 6, 2, 64, 16
    k, v, q = rows(rng, T, H, D), rows(rng, T, H, D), rows(rng, T, 4, D)
    cache = w4.PagedCache.make(3, kv.FMT[fmt], H, D, P)
    table = i32([[0, 1, -1, 3]])
    rope = w4.RopeTable(torch.ones(50, 32, 2, device="cuda"))
    # padding, fine, page -1, page 3 of 3, past the rotation table, fine
    pos = i32([-1, 5, 33, 49, 50, 31])
    qo = torch.full((T, 4, D), 9.0, device="cuda", dtype=torch.bfloat16)
    cache.append(to_gpu(k), to_gpu(v), pos, table, q=to_gpu(q), q_out=qo, rope=rope)
    torch.cuda.synchronize()
    assert cache.error.item() == w4.KV_ERR_PAGE | w4.KV_ERR_POSITION
    left = [0, 2, 3, 4]
    assert (qo[left] == 9.0).all() and not (qo[[1, 5]] == 9.0).all()
    with pytest.raises(w4.W4Error):
        cache.check()
    cache.check()                                            # cleared
    # sequences outside the table; positions past its width
    cache.append(to_gpu(k), to_gpu(v), i32([0, 1, 2, 3, 4, 64]), table,
                 seq_ids=i32([1, -1, 0, 0, 0, 0]))
    assert cache.error.item() == w4.KV_ERR_SEQUENCE | w4.KV_ERR_POSITION
    cache.error.zero_()
    got_k, got_v = cache.read(i32([2, 3, 4, -7, 33, 64]), table)
    assert np.array_equal(bits(got_k[:3]), kv.bf16_bits(kv.held(k[2:5], fmt)))
    assert (got_k[3:] == 0).all() and (got_v[3:] == 0).all()
    assert cache.error.item() == w4.KV_ERR_PAGE | w4.KV_ERR_POSITION
    # without an error word, and with no tokens at all
    cache._struct.error = None
    cache.append(to_gpu(k), to_gpu(v), i32([99] * 6), table)
    cache.append(to_gpu(k)[:0], to_gpu(v)[:0], i32([]), table)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_extreme_values(w4, fmt):
    """Infinite and NaN values, the largest and the smallest bfloat16s."""
    D, H = 128, 1
    x = np.zeros((8, H, D), np.float32)
    x[0, 0, 3], x[0, 0, 70] = np.inf, 1.0
    x[1, 0, 5], x[1, 0, 6] = -np.inf, 2.0
    x[2, 0, 7], x[2, 0, 8] = np.nan, -3.0
    x[3] = kv.bf16(np.full(D, 3e38, np.float32))
    x[4] = kv.bf16(np.full(D, 1e-38, np.float32))
    x[5, 0, :2] = kv.bf16(np.array([6e4, -6e4], np.float32))
    x[6, 0, 9] = kv.bf16(np.array([1e-6], np.float32))[0]
    x[7] = np.nan
    cache = w4.PagedCache.make(1, kv.FMT[fmt], H, D)
    table, pos = i32([[0]]), i32(np.arange(8))
    cache.append(to_gpu(x), to_gpu(x), pos, table)
    k, v = cache.read(pos, table)
    assert np.array_equal(bits(k), bits(v))
    got = k.float().cpu().numpy()
    if fmt == "bf16":
        assert np.array_equal(got, x, equal_nan=True)
        return
    assert np.isfinite(got).all()
    q = kv.LEVELS[fmt]
    assert got[0, 0, 3] == kv.bf16(np.float32(q * 65504)) and got[0, 0, 70] == 0
    assert got[1, 0, 5] == -kv.bf16(np.float32(q * 65504)) and got[1, 0, 6] == 0
    assert got[2, 0, 7] == 0 and got[2, 0, 8] < -2.9
    assert (got[3] == kv.bf16(np.float32(q * 65504))).all()
    assert (got[4] == 0).all() and (got[7] == 0).all()
    for i in (5, 6):
        assert np.array_equal(kv.bf16_bits(got[i]), kv.bf16_bits(kv.held(x[i], fmt)))


@pytest.mark.parametrize("fmt", list(kv.FMT))
def test_offsets_past_32_bits(w4, fmt):
    """Pages at the end of a pool of more than 4 GiB."""
    H, D, P = 4, 128, 16
    per_page = w4.kv_pool_bytes(kv.FMT[fmt], H, D, P, 1)
    pages = (5 << 30) // per_page
    if torch.cuda.mem_get_info()[0] < (7 << 30):
        pytest.skip("needs 7 GB")
    cache = w4.PagedCache(torch.empty(pages * per_page, dtype=torch.uint8, device="cuda"),
                          kv.FMT[fmt], H, D, P)
    rng = np.random.default_rng(2)
    k, v = rows(rng, 33, H, D), rows(rng, 33, H, D)
    table = i32([[pages - 1, 0, pages // 2 + 1]])
    cache.append(to_gpu(k), to_gpu(v), i32(np.arange(33)), table)
    k2, v2 = cache.read(i32(np.arange(33)), table)
    cache.check()
    assert np.array_equal(bits(k2), kv.bf16_bits(kv.held(k, fmt)))
    assert np.array_equal(bits(v2), kv.bf16_bits(kv.held(v, fmt)))
    tail = cache.pool[(pages - 1) * per_page:].cpu().numpy()
    host = kv.Pool(fmt, D, H, P, 1)
    for t in range(16):
        host.write(0, t, k[t], v[t])
    assert np.array_equal(tail, host.bytes.reshape(-1))


def test_refusals(w4):
    cache = w4.PagedCache.make(2, w4.KV_INT4, 2, 64)
    k = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    pos, table = i32([0, 1, 2, 3]), i32([[0, 1]])
    with pytest.raises(ValueError):
        cache.append(k[:, :1], k, pos, table)
    with pytest.raises(ValueError):
        cache.append(k, k, pos[:3], table)
    with pytest.raises(ValueError):
        cache.append(k, k, pos, table.long())
    with pytest.raises(ValueError):
        cache.append(k, k, pos, table, q=k)
    with pytest.raises(w4.W4Error) as e:
        cache.append(k[:3], k[:3], pos[:3], i32([[0], [1]]))       # 3 tokens of 2 sequences
    assert e.value.status == w4.Status.INVALID_ARG
    odd = torch.zeros(4 * 128 + 4, device="cuda", dtype=torch.bfloat16)[4:].view(4, 2, 64)
    for bad in ((odd, k), (k, odd)):
        with pytest.raises(w4.W4Error):
            cache.append(*bad, pos, table)
    with pytest.raises(w4.W4Error):
        cache.read(pos, table, k=odd)
    with pytest.raises(w4.W4Error):                                # not a multiple of 16
        cache.append(k, k, pos, table, rope=w4.RopeTable(torch.zeros(4, 4, 2, device="cuda")))
    with pytest.raises(ValueError):
        w4.PagedCache(torch.zeros(100, dtype=torch.uint8, device="cuda"), w4.KV_INT4, 2, 64)
    with pytest.raises(w4.W4Error):
        w4.PagedCache.make(2, w4.KV_INT4, 2, 96)
    with pytest.raises(w4.W4Error):
        w4.PagedCache.make(2, w4.KV_INT4, 2, 64, page_tokens=24)


@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("layout", [None, 0, 1])
def test_codes_of_many_values(w4, fmt, layout):
    """Every code of 4096 tokens: the scales that round the other way and the
    quotients next to a half, which small cases hardly meet."""
    rng = np.random.default_rng(7)
    T, H, D = 4096, 4, 128
    x, pos = rows(rng, T, H, D), np.arange(T, dtype=np.int32)
    table = torch.arange(T // 16, dtype=torch.int32, device="cuda").view(1, -1)
    rope, xr = None, x
    if layout is not None:
        angle = pos[:, None] * 1e6 ** (-np.arange(0, D, 2) / D)
        tab = np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)
        rope, xr = w4.RopeTable(torch.from_numpy(tab).cuda(), layout), kv.rotate(x, pos, tab, layout)
    cache = w4.PagedCache.make(T // 16, kv.FMT[fmt], H, D)
    cache.append(to_gpu(x), to_gpu(x), i32(pos), table, rope=rope)
    k, v = cache.read(i32(pos), table)
    assert np.array_equal(bits(k), kv.bf16_bits(kv.held(xr, fmt)))
    assert np.array_equal(bits(v), kv.bf16_bits(kv.held(x, fmt)))


@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("D,H,T", [(64, 2, 10007), (128, 4, 6003), (128, 1, 700), (64, 1, 333)])
def test_whole_records_and_others_agree(w4, fmt, D, H, T):
    """A run from inside a record on, long enough for a warp a record (or
    shorter, with four): its whole records are turned in shared memory; read
    back in reverse order, every token goes by itself."""
    rng = np.random.default_rng(T)
    first, P = 5, 32
    k, v = rows(rng, T, H, D), rows(rng, T, H, D)
    pos = np.arange(first, first + T, dtype=np.int32)
    pages = -(-(first + T) // P)
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda().view(1, -1)
    cache = w4.PagedCache.make(pages, kv.FMT[fmt], H, D, P)
    cache.append(to_gpu(k), to_gpu(v), i32(pos), table)
    forward = cache.read(i32(pos), table)
    backward = cache.read(i32(pos[::-1].copy()), table)
    cache.check()
    for x, got, turned in zip((k, v), forward, backward):
        want = kv.bf16_bits(kv.held(x, fmt))
        assert np.array_equal(bits(got), want)
        assert np.array_equal(bits(turned), want[::-1])
    # written in reverse, byte by byte: the same records
    again = w4.PagedCache.make(pages, kv.FMT[fmt], H, D, P)
    again.pool.zero_(), cache.pool.zero_()
    cache.append(to_gpu(k), to_gpu(v), i32(pos), table)
    back = pos[::-1].copy()
    again.append(to_gpu(k[::-1].copy()), to_gpu(v[::-1].copy()), i32(back), table)
    assert torch.equal(again.pool, cache.pool)
