"""Pages that finished requests give back (mxsa_build_tables): entries that are
no pages of the cache."""
import numpy as np
import pytest

from tests.test_gpu_tables import State, reference, refused, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("total", [500, 5000])  # one launch, two
@pytest.mark.parametrize("entry", [-1, -3, "pages", 2 ** 31 - 1])
def test_what_is_no_page_does_not_go_back(entry, total):
    s = State(np.random.RandomState(4), 9, 64, 700, spare=total // 64 + 2, extra=total // 64 + 20)
    assert min(s.held) > 0
    entry = s.pages if entry == "pages" else entry
    new = [3, -1, 0, -1, 1, 1, total - 40, -1, 5]
    want = reference(s.old, new, s.held, s.table, s.free, s.count, 64, total, s.pages)
    same(s.run(new, total), want)
    for row, at in ((1, 0), (7, s.held[7] - 1), (3, s.held[3] // 2)):
        page = s.table[row, at]
        s.table[row, at] = entry
        refused(s, new, total, 2048)
        s.table[row, at] = page
    # only what goes back is looked at: not the entries behind the held ones, nor a request's that held nothing
    s.table[1, s.held[1]:] = entry
    s.table[3] = entry
    s.held[3] = s.old[3] = 0
    want = reference(s.old, new, s.held, s.table, s.free, s.count, 64, total, s.pages)
    same(s.run(new, total), want)


def test_many_pages_of_which_the_last_is_none():
    """More pages than the plan has threads go back at once."""
    s = State(np.random.RandomState(7), 40, 64, 6000, extra=5)
    assert sum(s.held) > 1500
    same(s.run([-1] * 40, 8), reference(s.old, [-1] * 40, s.held, s.table, s.free, s.count, 64, 8, s.pages))
    s.table[39, s.held[39] - 1] = s.pages
    assert s.held[39] > 0
    refused(s, [-1] * 40, 8, 2048)
