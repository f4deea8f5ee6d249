"""Bad entries that the page operators report whatever else they have to do."""
import numpy as np
import pytest

from test_page_fork import Compact

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", ["moves", "no hole", "no moves allowed"])
@pytest.mark.parametrize("entry", [100, -2, 2 ** 31 - 1])
def test_a_bad_table_entry_is_reported_whether_pages_move_or_not(in_place, case, entry):
    c = Compact(100, [20, 30], 4, 40, 0 if case == "no moves allowed" else 50, in_place=in_place, shares=False)
    if case == "no hole":  # the same pool, its live pages the lowest
        to = np.empty(100, dtype=np.int32)
        live = [p for p in range(100) if p not in set(c.free)]
        to[live], to[c.free] = np.arange(len(live)), np.arange(len(live), 100)
        for b, k in enumerate((20, 30)):
            c.ttable[b * 40:b * 40 + k] = torch.from_numpy(to[c.table[b, :k]]).cuda()
        c.tfree[:len(c.free)] = torch.from_numpy(to[c.free]).cuda()
    before = c.ttable.clone()
    if case != "moves":
        c.run()
        torch.cuda.synchronize()
        assert int(c.err) == 0 and int(c.n[0]) == 0 and torch.equal(c.ttable, before)
    c.ttable[47] = entry
    c.ttable[25] = entry  # behind the first sequence's pages: not looked at
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == 32 and int(c.otable[47]) == entry and int(c.otable[25]) == entry
