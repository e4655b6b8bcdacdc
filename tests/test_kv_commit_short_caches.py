"""Caches and rings with fewer slots than the tree has nodes: bit-exact against the
sequential statement (a slot keeps the last token that is stored to it)."""
import pytest

from test_kv_commit_parity import check, w4  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,count,pos", [(4, 6, 0), (5, 8, 1), (1, 8, 0), (1, 8, 1)])
def test_full_cache(w4, T, count, pos):  # noqa: F811
    """A full cache never wraps: the first tokens stay, those past its end are refused."""
    assert check(w4, 20 + T, 2, 1, T, 8, 64, [[3, 0, 1, 7, 2, 6, 5, 4]], [count], [pos], False) == 1


@pytest.mark.parametrize("T,count,pos,bad", [(4, 9, 6, [8]), (4, 5, 0, [4]), (4, 9, 3, [4, 8]), (4, 9, 3, [0, 5]), (1, 9, 2, [8, 7]),
                                             (3, 8, 1, [0, 1, 2, 3, 4, 5, 6, 7]), (16, 9, 30, [2])])
def test_short_ring_with_refused_nodes(w4, T, count, pos, bad):  # noqa: F811
    """A refused token takes no slot: an earlier one that shares it stays."""
    path = [0, 1, 2, 3, 4, 5, 6, 7, 8]
    for i, j in enumerate(bad):
        path[j] = (-1, 9, -2 ** 31)[i % 3]
    assert check(w4, 30 + T, 2, 1, T, 9, 64, [path], [count], [pos], True) == 1


def test_short_ring_at_the_last_position(w4):  # noqa: F811
    """Positions past 2^31 - 1 are refused; the tokens before them keep their slots."""
    assert check(w4, 40, 1, 1, 4, 9, 64, [[0, 1, 2, 3, 4, 5, 6, 7, 8]], [6], [2 ** 31 - 3], True) == 1
