"""Attention over batches whose heads are cut close to their borders: two
blocks' cuts in one head, heads little longer than what is not cut off."""
import numpy as np
import pytest

from tests import kv_testutil as kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_paged_attn import Setup, run_both, w4  # noqa: E402, F401


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("lens", [[3360, 1200], [1200, 3360, 1200], [1200, 1216, 1232, 0, 1248]])
def test_heads_cut_near_their_borders(w4, fmt, lens):  # noqa: F811
    run_both(w4, Setup(w4, fmt, 128, 4, 7, 16, 1, lens, seed=len(lens)))


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D,H,group,M", [(128, 4, 7, 2), (128, 8, 4, 1), (64, 2, 7, 3),
                                         (128, 2, 8, 8)])
def test_ragged_batches_of_such_lengths(w4, fmt, D, H, group, M):  # noqa: F811
    rng = np.random.default_rng(D + H + M)
    for _ in range(3):
        lens = rng.integers(0, 2400, int(rng.integers(2, 9))).tolist()
        run_both(w4, Setup(w4, fmt, D, H, group, 16, M, lens, seed=M))
