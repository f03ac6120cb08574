"""w4_rope_table and w4_rope: the table against angles in exact integer
arithmetic, the rotation bit for bit against fp32 with one rounding an
operation and within its bound of fp64, the transposed map as a gradient, and
what is left out."""
import math
from fractions import Fraction

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


def randn(rng, *shape):
    return kv.bf16(rng.standard_normal(shape).astype(np.float32))


def to_gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(torch.bfloat16)


def frequencies(rot, base, scaling, factor, ctx, low, high):
    f = [float(base) ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == 1:
        return [x / factor for x in f]
    if scaling == 2:
        b = float(base) * factor ** (rot / (rot - 2))
        return [b ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == 3:
        keep = [min(1.0, max(0.0, (ctx * x / (2 * math.pi) - low) / (high - low))) for x in f]
        return [x * (g + (1 - g) / factor) for x, g in zip(f, keep)]
    return f


@pytest.mark.parametrize("rot,base,scaling,factor,amplitude", [
    (128, 1e6, 0, 1.0, 1.0), (64, 1e4, 1, 8.0, 1.0), (32, 1e4, 2, 4.0, 1.0),
    (128, 5e5, 3, 8.0, 1.0), (64, 1e4, 3, 4.0, 0.1 * math.log(4) + 1), (2, 1e4, 0, 1.0, 1.0),
    (6, 100.0, 0, 1.0, 0.5)])
def test_table(w4, rot, base, scaling, factor, amplitude):
    rows, ctx, low, high = 70001, 4096.0, 1.0, 32.0
    t = w4.RopeTable.make(rows, rot, base, scaling=scaling, factor=factor, original_context=ctx,
                          low_turns=low, high_turns=high, amplitude=amplitude).table.cpu().numpy()
    f = frequencies(rot, base, scaling, factor, ctx, low, high)
    # p * f (f a double, so its product with p is exact) modulo 2 pi: pi as a
    # rational good to 2^-140
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286,
                  10 ** 75)
    for p in (0, 1, 2, 777, 4096, 65537, rows - 1):
        for i in {0, 1, rot // 4, rot // 2 - 1} & set(range(rot // 2)):
            turns = Fraction(f[i]) / (2 * pi) * p
            angle = float((turns - round(turns)) * 2 * pi)
            want = np.array([math.cos(angle), math.sin(angle)]) * amplitude
            # the double-precision frequency may differ by 2^-50 relative
            # (pow on both sides), the fp32 result rounds by 2^-24 of itself
            tol = abs(amplitude) * (p * f[i] * 2.0 ** -50 + 2.0 ** -60) + 2.0 ** -24 * np.abs(want)
            assert (np.abs(t[p, i] - want) <= tol).all(), (p, i, t[p, i], want)


CASES = [  # tokens, heads, head_dim, rotary_dim
    (1, 1, 64, 64), (8, 32, 128, 128), (3, 16, 64, 32), (5, 7, 128, 16), (17, 3, 80, 20),
    (2, 5, 96, 24), (4, 2, 7, 6), (1, 1, 2, 2), (9, 40, 256, 128), (700, 3, 128, 64)]


@pytest.mark.parametrize("T,H,D,rot", CASES)
@pytest.mark.parametrize("layout", [0, 1])
def test_rotation(w4, T, H, D, rot, layout):
    rng = np.random.default_rng(T * 1000 + H + D + rot)
    table = rng.uniform(-1.5, 1.5, (1000, rot // 2, 2)).astype(np.float32)
    x = randn(rng, T, H, D)
    pos = rng.integers(0, 1000, T).astype(np.int32)
    pos[0], pos[-1] = 0, 999
    r = w4.RopeTable(torch.from_numpy(table).cuda(), layout)
    y = r.apply(to_gpu(x), torch.from_numpy(pos).cuda())
    torch.cuda.synchronize()
    want = kv.rotate(x, pos, table, layout)
    assert np.array_equal(bits(y), kv.bf16_bits(want))
    # fp64: three fp32 roundings of magnitudes up to |ac| + |bs|, one bf16 rounding
    ref = kv.rotate(x, pos, table, layout).astype(np.float64) * 0
    c, s = (table[pos][:, None, :, j].astype(np.float64) for j in (0, 1))
    n = rot // 2
    a, b = ((slice(0, n), slice(n, rot)) if layout == 0 else
            (slice(0, rot, 2), slice(1, rot, 2)))
    x64 = x.astype(np.float64)
    ref[...] = x64
    ref[..., a] = x64[..., a] * c - x64[..., b] * s
    ref[..., b] = x64[..., b] * c + x64[..., a] * s
    mag = np.abs(x64)
    mag[..., a] = np.abs(x64[..., a] * c) + np.abs(x64[..., b] * s)
    mag[..., b] = np.abs(x64[..., b] * c) + np.abs(x64[..., a] * s)
    got = y.float().cpu().numpy()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * mag).all()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T", [1, 6, 300])
def test_slices_in_place_and_odd_strides(w4, layout, T):
    """q and k of a fused row, in place; a head-major tensor; a row that starts
    on an odd element (no 16-byte accesses)."""
    rng = np.random.default_rng(T)
    D, H, rot = 128, 9, 128
    table = rng.uniform(-1, 1, (64, rot // 2, 2)).astype(np.float32)
    r = w4.RopeTable(torch.from_numpy(table).cuda(), layout)
    pos = rng.integers(0, 64, T).astype(np.int32)
    gpos = torch.from_numpy(pos).cuda()
    x = randn(rng, T, H + 2, D)
    want = kv.bf16_bits(kv.rotate(x[:, :H], pos, table, layout))
    rows = to_gpu(x)
    before = bits(rows[:, H:])
    out = rows[:, :H]
    assert r.apply(out, gpos, out=out).data_ptr() == rows.data_ptr()
    torch.cuda.synchronize()
    assert np.array_equal(bits(rows[:, :H]), want)
    assert np.array_equal(bits(rows[:, H:]), before)        # v is not touched
    head_major = to_gpu(x[:, :H].transpose(1, 0, 2)).transpose(0, 1)
    assert np.array_equal(bits(r.apply(head_major, gpos)), want)
    odd = torch.zeros(T * H * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H, D)
    odd.copy_(to_gpu(x[:, :H]))
    assert np.array_equal(bits(r.apply(odd, gpos, out=odd)), want)


def test_gradient(w4):
    """The transposed map: <g, R x> = <R^T g, x>, with R^T the call at the
    negative positions; and its entries against differences of the map."""
    rng = np.random.default_rng(3)
    T, H, D, rot = 5, 2, 64, 48
    table = rng.uniform(-1, 1, (50, rot // 2, 2)).astype(np.float32)
    pos = np.array([1, 7, 49, 20, 33], np.int32)
    for layout in (0, 1):
        r = w4.RopeTable(torch.from_numpy(table).cuda(), layout)
        g = randn(rng, T, H, D)
        back = r.apply(to_gpu(g), torch.from_numpy(-pos).cuda())
        # the map is linear: differences of it at unit steps are its columns
        want = np.zeros((T, H, D))
        for d in range(D):
            e = np.zeros((T, H, D), np.float32)
            e[..., d] = 1
            col = kv.rotate(e, pos, table, layout).astype(np.float64)
            want[..., d] = (col * g).sum(-1)
        got = back.float().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20).all()


def test_out_of_range_positions_are_left_out(w4):
    table = torch.rand(10, 32, 2, device="cuda")
    r = w4.RopeTable(table)
    x = torch.randn(5, 2, 64, device="cuda").to(torch.bfloat16)
    pos = torch.tensor([3, 10, -10, 9, 2147483647], dtype=torch.int32, device="cuda")
    y = torch.full_like(x, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r.apply(x, pos, out=y, error=err)
    r.apply(x, pos)                                   # without an error word
    torch.cuda.synchronize()
    assert err.item() == w4.KV_ERR_POSITION
    assert (y[[1, 2, 4]] == 7.0).all() and not (y[[0, 3]] == 7.0).any()
    lowest = torch.tensor([-2147483648] * 5, dtype=torch.int32, device="cuda")
    y.fill_(7.0)
    r.apply(x, lowest, out=y, error=err)
    assert (y == 7.0).all()


def test_no_tokens_and_other_stream(w4):
    r = w4.RopeTable(torch.rand(10, 32, 2, device="cuda"))
    none = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    r.apply(none, torch.empty(0, dtype=torch.int32, device="cuda"))
    x = torch.randn(64, 4, 64, device="cuda").to(torch.bfloat16)
    pos = torch.zeros(64, dtype=torch.int32, device="cuda")
    want = r.apply(x, pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = r.apply(x, pos, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals(w4):
    x = torch.zeros(2, 3, 64, device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    r = w4.RopeTable(torch.rand(10, 32, 2, device="cuda"))
    with pytest.raises(ValueError):
        r.apply(x.float(), pos)
    with pytest.raises(ValueError):
        r.apply(x, pos.long())
    with pytest.raises(ValueError):
        r.apply(x, pos[:1])
    with pytest.raises(ValueError):
        r.apply(x[..., ::2], pos)
    with pytest.raises(w4.W4Error):
        w4.RopeTable(torch.rand(10, 33, 2, device="cuda")).apply(x, pos)   # wider than a head
    with pytest.raises(w4.W4Error):
        w4.RopeTable(torch.rand(10, 32, 2, device="cuda"), 2).apply(x, pos)
