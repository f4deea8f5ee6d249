"""Shared attention over a workspace that earlier calls used: a call reads no partial result that it has not written itself."""
import numpy as np
import pytest

from test_shared_attention import TYPES, Call

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
COUNTERS = 16384  # bytes that are zero between calls


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def rows_behind(rows, shared, group=8):
    """Sequences of `rows` rows of a KV head (`group` heads) behind `shared` positions."""
    n = -(-rows // group)
    return [(shared, [shared + i % 5 for i in range(n)])]


def one_call(groups, nq, nkv, hd, page, io, cache, **kw):
    c = Call(groups, nq, nkv, hd, page, io, cache, **kw)
    c.ws[COUNTERS:].fill_(0xff)  # NaN, and numbers that are no place in a list
    c.run()
    c.check()
    assert not bool(c.ws[:COUNTERS].any())


# blocks of 129 to 256 rows are two numbers of the list of tiles, so short lists are cut between the two
@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f16")])
@pytest.mark.parametrize("rows,shared", [(136, 256), (136, 1000), (200, 384), (256, 700), (256, 2500), (256, 10000), (264, 1400), (384, 900), (392, 900)])
@pytest.mark.parametrize("nkv", [1, 2])
def test_lists_of_blocks_of_two_halves(io, cache, rows, shared, nkv):
    one_call(rows_behind(rows, shared), 8 * nkv, nkv, 64, 16, io, cache)


@pytest.mark.parametrize("io,cache", TYPES)
@pytest.mark.parametrize("groups,nq,nkv", [([(512, [513] * 32)], 28, 4), ([(2000, [2000 + i for i in range(32)])], 28, 4), ([(2500, [2500 + 3 * i for i in range(40)])], 12, 2),
                                           ([(300, [310] * 20), (0, [5, 0]), (1000, [1001] * 33), (64, [64])], 16, 2)])
def test_what_lies_in_the_workspace_is_not_read(io, cache, groups, nq, nkv):
    one_call(groups, nq, nkv, 128, 16, io, cache)


@pytest.mark.parametrize("hd,cache", [(256, "f16"), (256, "f32"), (64, "f32"), (16, "bf16")])
def test_what_lies_in_the_workspace_is_not_read_by_other_heads(hd, cache):
    one_call([(200, [201 + i for i in range(12)]), (0, [0, 300]), (1500, [1500])], 12, 2, hd, 16, "f32", cache)


def test_calls_of_other_groups_and_types_on_one_workspace():
    rng = np.random.default_rng(5)
    calls = []
    for i, (io, cache) in enumerate(TYPES * 3):
        n, shared = int(rng.integers(1, 60)), int(rng.integers(100, 4000))
        groups = [(shared, [shared + int(rng.integers(0, 50)) for _ in range(n)])] + [(0, [int(rng.integers(0, 400))])] * int(rng.integers(0, 4))
        # scores far below zero, so that a state of another call, or one of zeros, would win over all of them
        calls.append(Call(groups, 16, 2, (64, 128)[i % 2], 16, io, cache, seed=i))
        c = calls[-1]
        c.tq[:n] = c.tq[:n].abs() * 4
        for arr, t in ((c.c.k, c.c.tk),):
            t.copy_(-t.abs() * 4)
            for b, x in enumerate(arr):
                arr[b] = -np.abs(x) * 4
    ws = torch.zeros(max(c.ws.numel() for c in calls), dtype=torch.uint8, device="cuda")
    for c in calls:
        c.ws = ws
    for turn in range(3):
        for i in rng.permutation(len(calls)):
            calls[i].out.fill_(3.0)
            calls[i].lse.fill_(3.0)
            calls[i].run()
            calls[i].check()
