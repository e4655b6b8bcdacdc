"""Caches and rings with fewer slots than the tree has nodes: bit-exact against the
sequential statement (a slot keeps the last token that is stored to it)."""
import pytest

from test_kv_commit_parity import check, w4  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,count,pos", [(4, 6, 0), (5, 8, 1), (1, 8, 0), (1, 8, 1)])
def test_full_cache(w4, T, count, pos):  # noqa: F811
    """A full cache never wraps: the first tokens stay, those past its end are refused."""
    assert check(w4, 20 + T, 2, 1, T, 8, 64, [[3, 0, 1, 7, 2, 6, 5, 4]], [count], [pos], False) == 1
