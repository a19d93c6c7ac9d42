"""Reorders over tables that list a page more often than its count of holders says: the whole call is refused,
whichever of the holders goes, stays or has children, and nothing changes."""
import pytest
import torch

from test_gpu_pages import DEV, Cache, kvc, state, unchanged  # noqa: F401

pytestmark = pytest.mark.gpu
# tables that one block and a cluster take
TABLES = pytest.mark.parametrize("mb", [12, 2100])
PARENTS = [[-1, 1, 2], [0, -1, 2], [-1, 0, 2], [0, 0, 2], [1, 1, 2], [1, -1, 2], [1, 0, 2], [2, 1, 2], [-1, -1, 2], [0, 1, 2],
           [0, 1, 0], [-1, -1, -1], [2, 2, 2]]


def refused(c, parent, code=9):
    before = state(c)
    c.kvc.kvc_pages_reorder(c.pool, c.pt, c.free, c.shares, torch.tensor(parent, dtype=torch.int32, device=DEV), pos=c.pos)
    assert c.kvc.kvc_device_status() == code
    unchanged(c, before)


@TABLES
@pytest.mark.parametrize("parent", PARENTS)
def test_a_page_of_two_tables_counted_once(kvc, mb, parent):  # noqa: F811
    c = Cache(kvc, [40, 32, 5], max_blocks=mb)
    c.table[1, 0] = c.table[0, 1]
    refused(c, parent)


@TABLES
@pytest.mark.parametrize("parent", PARENTS)
def test_a_page_twice_in_a_table(kvc, mb, parent):  # noqa: F811
    c = Cache(kvc, [32, 48, 5], max_blocks=mb)
    c.table[1, 2] = c.table[1, 0]
    refused(c, parent)


@TABLES
@pytest.mark.parametrize("parent", [p for p in PARENTS])
def test_a_page_of_three_tables_counted_twice(kvc, mb, parent):  # noqa: F811
    c = Cache(kvc, [32, 33, 16], max_blocks=mb)
    c.table[1, 0] = c.table[2, 0] = c.table[0, 1]
    c.shares[c.table[0, 1].long()] = 1
    refused(c, parent)


@TABLES
@pytest.mark.parametrize("parent", [[-1, 1, 2], [0, 0, 2], [-1, 0, 2], [0, 1, 2]])
def test_a_partly_filled_page_of_two_tables(kvc, mb, parent):  # noqa: F811
    c = Cache(kvc, [40, 24, 5], max_blocks=mb)
    c.table[1, 1] = c.table[0, 2]
    refused(c, parent)


@TABLES
@pytest.mark.parametrize("listed", [True, False])
def test_counts_below_zero(kvc, mb, listed):  # noqa: F811
    c = Cache(kvc, [40, 32, 5], max_blocks=mb)
    c.shares[c.table[1, 0].long() if listed else c.ids[0].long()] = -1
    refused(c, [0, 0, 2])


@TABLES
def test_an_id_outside_the_pool_of_a_sequence_that_stays(kvc, mb):  # noqa: F811
    c = Cache(kvc, [40, 32, 5], max_blocks=mb)
    c.table[2, 0] = c.k.shape[1]
    refused(c, [0, 0, 2])
    c.table[2, 0] = -1
    refused(c, [0, 0, 2])


@TABLES
def test_holders_outside_the_tables(kvc, mb):  # noqa: F811
    """A page may be counted more often than it is listed: someone else holds it, and it is not freed."""
    c = Cache(kvc, [32, 40, 5], max_blocks=mb)
    kept = int(c.table[0, 1])
    c.shares[kept] = 2
    c.model.shares[kept] = 2
    for parent in ([-1, 1, 1], [1, 1, 1]):
        c.reorder(parent)
        assert kvc.kvc_device_status() == 0
        c.model.same_as(c.table, c.n_blocks, c.len, c.score, c.ids, c.top, c.shares)
    assert int(c.shares[kept]) == 1 and kept not in c.ids[:int(c.top)].tolist()


@TABLES
def test_sequences_that_stay_keep_their_pages(kvc, mb):  # noqa: F811
    """Properly counted pages: one holder goes, one has children, one stays."""
    c = Cache(kvc, [50, 0, 0, 0, 17], max_blocks=mb)
    c.reorder([0, 0, 0, 0, 4])
    for parent in ([0, 1, -1, 1, 4], [0, -1, 2, 3, 3], [0, 0, 2, -1, 4], [-1, 1, -1, -1, -1], [-1] * 5):
        c.reorder(parent)
        assert kvc.kvc_device_status() == 0
        c.check()


@pytest.mark.parametrize("NB", [32, 33, 34, 35])
def test_pools_of_odd_and_even_sizes(kvc, NB):  # noqa: F811
    """The counts of a pool's pages lie in the workspace before the tables that follow them."""
    c = Cache(kvc, [50, 30, 16, 3], spare=NB - 8, max_blocks=2100)
    assert c.k.shape[1] == NB
    ws = kvc.pages_workspace(4, 2100, NB, DEV)
    ws.fill_(0xAB)
    for parent in ([1, 1, 0, 0], [3, 3, 2, -1], [0, 0, 0, 1]):
        c.reorder(parent, ws=ws)
        assert kvc.kvc_device_status() == 0
        c.check()
