"""w4_select with more rows than the device has multiprocessors, at the row lengths
where its variants for many rows begin and end: one block of 512 threads a row, then
clusters of which not all run at a time, then one block of 1024 threads."""
import numpy as np
import pytest

from tests.test_gpu_select import check, w4  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def ragged(rng, B, columns):
    lens = rng.integers(columns // 2, columns + 1, B)
    lens[:6] = columns, columns - 1, 1, 0, columns // 3, 4096
    return lens.tolist()


@pytest.mark.parametrize("columns", [4096, 4097, 8191, 8192, 8193, 16384, 16385])
@pytest.mark.parametrize("kind", ["normal", "equal", "few", "special"])
def test_more_rows_than_multiprocessors(w4, columns, kind):  # noqa: F811
    rng = np.random.default_rng(columns + len(kind))
    B, H = 77, 4                                          # 308 rows
    shape = (B, H, columns)
    x = {
        "normal": lambda: rng.standard_normal(shape),
        "equal": lambda: np.full(shape, -2.25),
        "few": lambda: rng.integers(0, 3, shape),
        "special": lambda: rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1.0], shape),
    }[kind]().astype(np.float32)
    lens = ragged(rng, B, columns)
    check(w4, x, lens, 64, first=4, last=16)
    check(w4, x, lens, 1)
    check(w4, x, lens, columns // 4)
    check(w4, x, lens, columns - 1, first=columns // 2, last=5)


@pytest.mark.parametrize("columns", [24576, 24577, 32768, 32769])
def test_many_rows_of_a_block_each(w4, columns):  # noqa: F811
    rng = np.random.default_rng(columns)
    lens = ragged(rng, 40, columns)
    x = rng.standard_normal((40, 4, columns)).astype(np.float32)
    check(w4, x, lens, 4096, first=4, last=128)
    check(w4, np.round(x), lens, 900)


def test_units_of_many_rows(w4):  # noqa: F811
    """Items of 16 tokens, lengths past the columns among them."""
    rng = np.random.default_rng(7)
    lens = [16 * n + int(d) for n, d in zip(ragged(rng, 90, 8000), rng.integers(0, 16, 90))]
    lens[7:9] = 10 ** 6, 2 ** 31 - 1
    check(w4, rng.standard_normal((90, 2, 8000)).astype(np.float32), lens, 500, unit=16, first=1,
          last=2)
