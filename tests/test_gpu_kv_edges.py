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
