"""w4_sparse_attn over one sequence at list lengths around those from which a head's
records are shared by blocks and joined by a second launch: every output is written
(what was there before is a mark), and right against fp64."""
import numpy as np
import pytest

from tests import kv_testutil as kv
from tests.test_gpu_paged_attn import Setup, i32
from tests.test_gpu_sparse_attn import check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# Per new-token count, listed records of 16 tokens: on both sides of the first length at
# which a listed head is cut, and of the one from which the whole attention's would be.
WIDE = {1: (77, 78, 103, 104), 2: (49, 50, 55, 56), 3: (24, 25, 31, 32), 4: (29, 30, 39, 40),
        8: (12, 13, 15, 16)}
NARROW = {1: (79, 80, 119, 120, 143, 144), 2: (53, 54, 71, 72), 3: (35, 36, 47, 48),
          4: (39, 40, 55, 56), 8: (17, 18, 23, 24)}
SHAPES = [("int8", 128, 4, 7, WIDE), ("int4", 128, 4, 7, {**WIDE, 1: (79, 80, 111, 112)}),
          ("bf16", 128, 4, 7, WIDE), ("bf16", 64, 2, 7, NARROW), ("int8", 64, 2, 7, NARROW),
          ("int4", 64, 2, 7, NARROW)]
MARK = 777.0


@pytest.fixture(scope="module")
def w4():
    from int4_weight_only_w4_gb300 import w4 as mod
    return mod


def run_marked(w4, s, P, blocks, counts):
    """Both calls on outputs that hold a mark."""
    gb, gc = i32(blocks), i32(counts)
    chosen = [[row[:c] for row in seq] for seq, c in zip(blocks, counts)]
    results = []
    for fn, dtype in ((w4.sparse_attn, torch.bfloat16), (w4.sparse_attn_f32, torch.float32)):
        out = torch.full(s.gq.shape, MARK, device="cuda", dtype=dtype)
        lse = torch.full(s.gq.shape[:2], MARK, device="cuda")
        ws = torch.full_like(s.cache.new_workspace(), 0xFF)
        fn(s.cache, s.gq, out, s.glens, s.table, gb, gc, ws, lse=lse)
        check(s, out, lse, P, chosen, bf16_out=dtype is torch.bfloat16, what=str(dtype))
        results.append((out, lse))
    (a, lse), (b, lse32) = results
    assert torch.equal(b.to(torch.bfloat16), a) and torch.equal(lse, lse32)


@pytest.mark.parametrize("fmt,D,H,group,counts", SHAPES)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 8])
def test_one_sequence(w4, fmt, D, H, group, counts, M):
    top = max(counts[M]) + 3
    s = Setup(w4, fmt, D, H, group, 16, M, [16 * top - 5], seed=D + M)
    rng = np.random.default_rng(M)
    for n in counts[M]:
        blocks = np.stack([np.sort(rng.permutation(top)[:n]) for _ in range(H)])[None]
        run_marked(w4, s, 16, blocks, [n])                # the list's room is its count,
        wider = np.full((1, H, n + 5), -1)
        wider[:, :, :n] = blocks
        run_marked(w4, s, 16, wider, [n])                 # or more
    s.cache.check()


@pytest.mark.parametrize("fmt,blocks", [("int8", 20), ("int8", 25), ("int4", 27), ("int8", 26)])
def test_one_sequence_in_pages_of_64(w4, fmt, blocks):
    s = Setup(w4, fmt, 128, 4, 7, 64, 1, [64 * 30 - 11], seed=blocks)
    rng = np.random.default_rng(blocks)
    index = np.stack([np.sort(rng.permutation(30)[:blocks]) for _ in range(4)])[None]
    run_marked(w4, s, 64, index, [blocks])
    s.cache.check()


def test_a_count_below_the_room(w4):
    """The room of the list, not its count, decides whether the joining launch is made:
    lists that are cut in wide rooms, and lists that are not."""
    s = Setup(w4, "int8", 128, 2, 7, 16, 1, [16 * 110], seed=1)
    for n in (0, 1, 60, 78, 100):
        index = np.tile(np.arange(200), (1, 2, 1))
        run_marked(w4, s, 16, index, [n])
    s.cache.check()
