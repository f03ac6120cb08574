"""Bounds of pages that several sequences share: those of their tokens where the page
holds as many in each of the sequences, whichever of them is the last to write."""
import numpy as np
import pytest

from tests import kv_testutil as kv
from tests.test_gpu_key_blocks import check_scores, host, want_scores
from tests.test_gpu_paged_attn import Setup, i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def w4():
    from int4_weight_only_w4_gb300 import w4 as mod
    return mod


@pytest.mark.parametrize("fmt", list(kv.FMT))
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (128, 32)])
def test_a_shared_prompt(w4, fmt, D, P):
    """Forty sequences over the pages of one: full ones, and a last one that holds the
    same tokens in some and is not reached by the others."""
    n, H = 5 * P + 9, 2
    s = Setup(w4, fmt, D, H, 3, P, 1, [n], seed=P)
    B = 40
    lens = [n if b % 3 else 5 * P - P * (b % 2) for b in range(B)]
    table, glens = s.table.expand(B, -1).contiguous(), i32(lens)
    k = kv.bf16(s.keys[0])
    want = np.zeros(s.cache.bounds_shape, np.float32)
    for i, page in enumerate(s.table[0].cpu().numpy()[:6]):
        part = k[i * P:min(n, i * P + P)]
        want[page, :, 0], want[page, :, 1] = part.max(0), part.min(0)
    q = torch.randn(B, 3 * H, D, device="cuda").to(torch.bfloat16)
    for _ in range(5):
        bounds = s.cache.new_bounds()
        s.cache.key_bounds(bounds, glens, table, tokens=10 ** 6)
        assert np.array_equal(host(bounds), want)
    scores = s.cache.block_scores(bounds, q, glens, table)
    plain, mag = want_scores(want, host(q), lens, 1, table.cpu().numpy(), P, H, table.shape[1])
    there = np.arange(table.shape[1]) < -(-np.array(lens) // P)[:, None]
    there = np.broadcast_to(there[:, None], plain.shape)
    check_scores(host(scores)[there], plain[there], mag[there], D)
    assert np.isneginf(host(scores)[~there]).all()
    s.cache.check()
