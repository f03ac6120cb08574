"""w4_select against a stable sort on the host: exact, whatever the scores are
(equal ones, both zeros, infinities, NaN), at row lengths around every border of
the kernels' variants, with the first and last items kept."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

MARK = -9


@pytest.fixture(scope="module")
def w4():
    from int4_weight_only_w4_gb300 import w4 as mod
    return mod


def plain(scores, n, first, last, count):
    """The chosen ones of the first n scores."""
    if n <= count:
        return np.arange(n)
    always = np.zeros(n, bool)
    always[:first] = True
    always[n - last:] = True
    x = scores[:n].astype(np.float64)
    # by: always, NaN, score; a stable sort keeps the order of equal ones
    order = np.lexsort((np.where(np.isnan(x), 0, -x), ~np.isnan(x), ~always))
    return np.sort(order[:count])


def check(w4, scores, lens, count, unit=1, first=0, last=0, **kw):
    B, H, columns = scores.shape
    gs = torch.from_numpy(scores).cuda()
    gl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    index = torch.full((B, H, count), MARK, dtype=torch.int32, device="cuda")
    counts = torch.full((B,), MARK, dtype=torch.int32, device="cuda")
    w4.select(gs, gl, index, counts, unit=unit, first=first, last=last, **kw)
    torch.cuda.synchronize()
    got = index.cpu().numpy()
    for b, n in enumerate(lens):
        n = min(-(-max(n, 0) // unit), columns)
        assert counts[b].item() == min(n, count)
        for h in range(H):
            want = np.full(count, MARK)
            chosen = plain(scores[b, h], n, first, last, count)
            want[:len(chosen)] = chosen
            assert np.array_equal(got[b, h], want), (b, h, n, count)
    return gs, gl, index, counts


@pytest.mark.parametrize("columns", [1, 2, 31, 33, 255, 257, 1000, 4095, 4096, 4097, 8191, 16384,
                                     16385, 32768, 32769, 65537, 131072, 131073, 200001, 262144,
                                     262145, 300001])
def test_row_lengths(w4, columns):
    rng = np.random.default_rng(columns)
    B, H = (5, 3) if columns < 20000 else (2, 2)
    scores = rng.standard_normal((B, H, columns)).astype(np.float32)
    lens = [columns] + [int(x) for x in rng.integers(0, columns + 1, B - 1)]
    for count in sorted({1, 2, min(64, columns), max(1, columns // 8), max(1, columns - 1),
                         columns, columns + 5}):
        check(w4, scores, lens, count)
        check(w4, scores, lens, count, first=min(4, count // 2), last=count // 3)


@pytest.mark.parametrize("columns", [700, 3000, 9000, 40000, 150000, 270000])
@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "special", "decades", "negative",
                                  "close"])
def test_score_values(w4, columns, kind):
    rng = np.random.default_rng(len(kind) + columns)
    shape = (2, 2, columns)
    x = {
        "equal": lambda: np.full(shape, 3.5),
        "few": lambda: rng.integers(0, 3, shape),
        "zeros": lambda: rng.choice([0.0, -0.0], shape),
        "special": lambda: rng.choice([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45,
                                       3e38, -3e38], shape),
        "decades": lambda: np.where(rng.random(shape) < 0.1, 0,
                                    np.exp(3 * rng.standard_normal(shape) - 8)),
        "negative": lambda: -np.abs(rng.standard_normal(shape)) - 1,
        # neighbours in fp32: told apart by their last digit only
        "close": lambda: (rng.integers(0, 5, shape) + 0x3F800000).astype(np.uint32).view(
            np.float32),
    }[kind]()
    x = np.ascontiguousarray(x, np.float32)
    for count in (1, 77, columns // 3, columns - 1):
        check(w4, x, [columns, columns - 50], count)
        check(w4, x, [columns, columns - 50], count, first=count // 4, last=count // 2)


def test_units_and_lengths(w4):
    rng = np.random.default_rng(0)
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 800, 1599, 1600, 1601, 10 ** 6, 2 ** 31 - 1, -7]
    scores = rng.standard_normal((len(lens), 2, 100)).astype(np.float32)
    check(w4, scores, lens, 10, unit=16, first=1, last=2)
    check(w4, scores, lens, 10, unit=1, first=10)
    check(w4, scores, lens, 10, unit=2 ** 31 - 1, last=10)


def test_always_chosen_meet_nan(w4):
    """The first and last items stay whatever the others are."""
    x = np.full((1, 1, 5000), np.nan, np.float32)
    check(w4, x, [5000], 40, first=7, last=20)
    check(w4, x, [5000], 27, first=7, last=20)


def test_many_rows(w4):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 300, 500).tolist()
    check(w4, rng.standard_normal((500, 4, 300)).astype(np.float32), lens, 16, first=1, last=2)


def test_many_long_rows(w4):
    """More rows than the device has clusters for at a time."""
    rng = np.random.default_rng(5)
    lens = rng.integers(9000, 40001, 60).tolist()
    check(w4, rng.integers(0, 9000, (60, 2, 40000)).astype(np.float32), lens, 700, first=1, last=2)


def test_stream_graph_and_repeats(w4):
    rng = np.random.default_rng(2)
    x = rng.integers(0, 50, (3, 2, 30000)).astype(np.float32)
    gs, gl, index, counts = check(w4, x, [30000, 100, 20000], 500, last=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(w4, x, [30000, 100, 20000], 500, last=9, stream=side)
    again, n = torch.empty_like(index), torch.empty_like(counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.select(gs, gl, again, n, last=9)
    for _ in range(20):
        again.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, index) and torch.equal(n, counts)


def test_refusals(w4):
    s = torch.zeros(2, 3, 40, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    index = torch.zeros(2, 3, 8, dtype=torch.int32, device="cuda")
    w4.select(s, lens, index, lens.clone())
    for a in ((s[0], lens, index, lens), (s.double(), lens, index, lens),
              (s, lens[:1], index, lens), (s, lens, index[:, :2], lens),
              (s, lens, index.long(), lens), (s.transpose(1, 2), lens, index, lens),
              (s, lens, index, lens[:1]), (s.cpu(), lens, index, lens)):
        with pytest.raises(ValueError):
            w4.select(*a)
    for kw in (dict(unit=0), dict(first=-1), dict(last=-1), dict(first=5, last=4)):
        with pytest.raises(w4.W4Error) as e:
            w4.select(s, lens, index, lens.clone(), **kw)
        assert e.value.status == w4.Status.INVALID_ARG
