"""Tables in which a row names a page more than once, as where unused places hold one page that stands for none:
a call that writes them leaves no page with two places."""
import numpy as np
import pytest

from gpu_util import to_dev_i32
from test_cache_pages_gpu import GUARD, ints, reserve, tsd  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def run(tsd, table, counts, lens, new, page=16):  # noqa: F811
    t, c = to_dev_i32(np.array(table)), to_dev_i32(np.array(counts))
    copies, n, missing = reserve(tsd, t, c, to_dev_i32(lens), to_dev_i32(new), int(max(new)), page)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK and (copies[n:] == GUARD).all()
    t, c = ints(t), ints(c)
    assert np.array_equal(c, np.bincount(t[t >= 0], minlength=len(c)))
    return t.tolist(), c.tolist(), copies[:n].tolist(), missing


def test_one_row(tsd):  # noqa: F811
    """Both places written: the first keeps the page. With earlier tokens in it, too; and where the first is not written,
    the second is a copy of nothing or of what lies ahead of the new tokens."""
    assert run(tsd, [[0, 0, -1]], [2, 0, 0, 0], [32], [32])[:3] == ([[0, 1, -1]], [1, 1, 0, 0], [])
    assert run(tsd, [[0, 0, -1]], [2, 0, 0, 0], [40], [30])[:3] == ([[0, 1, 2]], [1, 1, 1, 0], [])
    assert run(tsd, [[0, 0, 0]], [3, 0, 0, 0], [48], [32])[:3] == ([[0, 1, 2]], [1, 1, 1, 0], [])
    assert run(tsd, [[0, 0, 0]], [3, 0, 0, 0], [48], [30])[:3] == ([[0, 1, 2]], [1, 1, 1, 0], [[0, 1, 2]])


def test_several_rows(tsd):  # noqa: F811
    """The first place of the first row that writes it keeps the page, the others leave it; one that another row
    holds without writing it is kept by nobody."""
    table = [[-1, 0], [0, 0], [1, 0]]
    assert run(tsd, table, [4, 1, 0, 0, 0, 0, 0], [32, 32, 32], [32, 28, 28])[:3] == (
        [[2, 0], [3, 4], [1, 5]], [1] * 6 + [0], [[0, 3, 4]])
    table = [[-1, 2], [2, 2], [2, -1]]
    assert run(tsd, table, [0, 0, 4, 0, 0, 0, 0], [16, 32, 0], [16, 28, 0])[:3] == (
        [[0, 2], [1, 3], [2, -1]], [1, 1, 2, 1, 0, 0, 0], [[2, 1, 4]])


@pytest.mark.parametrize("B,pages", [(1, 40), (3, 70), (40, 33), (1000, 17), (30000, 2)])
def test_one_page_for_all_places(tsd, B, pages):  # noqa: F811
    """Every place of every row names page 5: the first keeps it, the lowest free ones go to the others in order;
    one block and several, a place to a thread and many."""
    need = B * pages
    counts = np.zeros(need + 3, int)
    counts[5] = need
    t, c, copies, missing = run(tsd, np.full((B, pages), 5), counts, [pages * 16] * B, [pages * 16] * B)
    assert (copies, missing) == ([], 0)
    assert np.array_equal(np.ravel(t), np.append(5, np.delete(np.arange(need), 5)))
    assert c == [1] * need + [0] * 3


@pytest.mark.parametrize("B,pages", [(1, 4), (2, 40), (3000, 8)])
def test_short_of_pages(tsd, B, pages):  # noqa: F811
    """One page too few: everything as it was."""
    need = B * pages
    counts = np.zeros(max(need - 1, 2), int)
    counts[1] = need
    t, c, copies, missing = run(tsd, np.full((B, pages), 1), counts, [pages * 16] * B, [pages * 16 - 3] * B)
    assert (copies, missing) == ([], 1) and np.array_equal(t, np.full((B, pages), 1)) and c == counts.tolist()
