"""Tables whose room comes close to 2^31 tokens: refused on the host where a length and
what the kernels add to it would leave 32 bits.  (Every call here fails validation, the
allowed sizes by another argument that is checked later, so no pointer is looked at.)"""
import pytest

from tests.test_abi_host import FAKE, lib  # noqa: F401
from tests.test_kv_host import cache, table
from tests.test_long_host import bounds, gather, scores, sparse, weights

ROOM = 2 ** 31 - 2 ** 21                # the most of the calls that walk all sequences


def sized(page, room, pages=FAKE):
    """A cache and a table of one sequence with this room."""
    assert room % page == 0
    return cache(kv_heads=1, page_tokens=page), table(pages, width=room // page,
                                                      stride=room // page)


def walks(lib, page, room, late):  # noqa: F811
    """All calls that walk the sequences; late: with an argument that is refused after
    the sizes."""
    c, t = sized(page, room)
    kw = dict(c=c, t=t)
    yield bounds(lib, **kw, **(dict(out=None) if late else {}))
    yield scores(lib, **kw, hq=1, columns=1 << 28, **(dict(b=None) if late else {}))
    yield weights(lib, **kw, hq=1, columns=1 << 30, **(dict(lse=None) if late else {}))
    yield gather(lib, **kw, to=table(FAKE + 64), **(dict(index=None) if late else {}))
    # the room of the new places
    yield gather(lib, c=c, t=table(), to=sized(page, room, FAKE + 64)[1],
                 **(dict(index=None) if late else {}))


@pytest.mark.parametrize("page", [16, 48, 64, 1 << 20])
def test_walks_refuse_rooms_near_the_limit(lib, page):  # noqa: F811
    for room in (2 ** 31 - 1, 2 ** 31 - 2 ** 20, ROOM + page):
        room -= room % page
        assert room > ROOM
        assert list(walks(lib, page, room, False)) == [2] * 5


@pytest.mark.parametrize("page", [16, 48, 64, 1 << 20])
def test_walks_allow_what_is_below(lib, page):  # noqa: F811
    assert list(walks(lib, page, ROOM - ROOM % page, True)) == [1] * 5
