"""The paged attention within the close bounds of attn_bounds.py: results and
log-sum-exps of every format, head size and form of the call."""
import numpy as np
import pytest

from tests import attn_bounds as ab

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_paged_attn import Setup, w4  # noqa: E402, F401


def both(w4, s, scale, window, what):  # noqa: F811
    codes = None
    if s.fmt != "bf16":
        table = s.table.cpu().numpy()
        codes = [ab.pool_codes(s.host, table[b], n) for b, n in enumerate(s.lens)]
    rows = ab.rows_of(s.fmt, s.q, s.keys, s.values, codes, s.lens, s.M, scale, window)
    out = torch.empty(s.gq.shape, device="cuda")
    lse = torch.empty(s.gq.shape[:2], device="cuda")
    w4.paged_attn_f32(s.cache, s.gq, out, s.glens, s.table, s.cache.new_workspace(), scale, window,
                      lse)
    ab.check(out.cpu().numpy(), lse.cpu().numpy(), rows, s.fmt, False, what + " fp32")
    got, lse = s.cache.attend(s.gq, s.glens, s.table, scale=scale, window=window)
    ab.check(got.float().cpu().numpy(), lse.cpu().numpy(), rows, s.fmt, True, what + " bf16")
    s.cache.check()


@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("D,H,group,P", [(128, 4, 7, 16), (64, 2, 7, 32), (64, 3, 5, 48)])
@pytest.mark.parametrize("M", [1, 3, 8])
def test_formats_heads_and_windows(w4, fmt, D, H, group, P, M):  # noqa: F811
    s = Setup(w4, fmt, D, H, group, P, M, [0, 1, 17, 64, 500, 1300], seed=D + H + M)
    for scale, window in ((D ** -0.5, 0), (-0.07, 100)):
        both(w4, s, scale, window, f"scale {scale} window {window}")


@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_keys_of_other_sizes(w4, fmt):  # noqa: F811
    """Keys far smaller or larger than the queries, with the scale that makes up
    for it."""
    rng = np.random.default_rng(5)
    for power in (-6, 3):
        s = Setup(w4, fmt, 128, 2, 4, 16, 2, [40, 700], seed=power + 20, spread=2.0 ** power)
        both(w4, s, 128 ** -0.5 * 2.0 ** -power * rng.uniform(0.5, 1), 0, f"2^{power}")
