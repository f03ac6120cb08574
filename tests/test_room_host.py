"""Tables whose room comes close to 2^31 tokens: refused on the host where a length and
what the kernels add to it would leave 32 bits.  (Every call here fails validation, the
allowed sizes by another argument that is checked later, so no pointer is looked at.)"""
import pytest

from tests.test_abi_host import FAKE, lib  # noqa: F401
from tests.test_kv_host import attn, cache, table
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


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_attention(lib, page, listed, f32):  # noqa: F811
    """A record that is not there (its page is bad, or it lies past the end of a listed
    block) counts as one behind key 2^31 - 256: no sequence may be longer than that."""
    def call(room):
        c, t = sized(page, room - room % page)
        if listed:
            return sparse(lib, name="w4_sparse_attn" + ("_f32" if f32 else ""), c=c, t=t, hq=1)
        return attn(lib, c=c, t=t, hq=1, f32=f32, n=0)

    for room in (2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 240):
        assert (call(room) == 2) == (room - room % page > 2 ** 31 - 256), room
    # (a workspace of no bytes is refused last, with a device; without one its size is not known)
    assert call(2 ** 31 - 256) in (1, 4)
