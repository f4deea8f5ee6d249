"""A page that sequences hold although it is on the free list: a fork that ends them would put it there a second time."""
import pytest

from test_page_fork import Fork, Pool, taken

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("in_place", [False, True])
def test_more_free_pages_than_the_pool_has_are_reported_as_pages(in_place):
    pool = Pool([[9, 5], [6]], 4, 4, spare=0)
    n = pool.n_pages
    pool.free = list(range(n))  # every page, those of the sequences too
    f = Fork(pool, [0, -1], in_place=in_place)
    f.run()
    torch.cuda.synchronize()
    assert int(f.err) == 32                               # not the error of a fork that was refused:
    assert taken(f.lens, 2).tolist() == [9, 0]            # it was carried out
    assert int(f.n[0]) == n and taken(f.free, n).tolist() == list(range(n))
    assert not bool(f.ws[12:].any())
