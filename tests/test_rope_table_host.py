"""w4_rope_table refuses frequencies that are not finite, on the host: each part
of the specification is finite by itself, together they are not."""
import pytest

from tests.test_abi_host import FAKE, lib  # noqa: F401
from tests.test_kv_host import P, I, ref, spec


@pytest.mark.parametrize("kw", [
    dict(scaling=1, base=1e-300, factor=1e-200),            # f / factor
    dict(scaling=2, base=1e4, factor=1e-300, rotary_dim=4),  # base * 0
    dict(scaling=2, base=1e300, factor=1e300),              # base * inf
    dict(scaling=3, base=1e-300, factor=1e-200, original_context=4096.0, low_turns=1.0,
         high_turns=1e308)])
def test_frequencies_that_are_not_finite(lib, kw):  # noqa: F811
    lib.w4_rope_table.argtypes = [P, I, P, P]
    assert lib.w4_rope_table(ref(spec(**kw)), 10, FAKE, None) == 1
