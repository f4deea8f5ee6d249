"""Forks of sequences over counted pages, copies of pages and compaction of the pool, on the GPU against loops:
whole numbers and moved bits, so equal."""
import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
GUARD = -77  # behind every output


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def guarded(n):
    return torch.full((n + 3,), GUARD, dtype=torch.int32, device="cuda")


def taken(t, n):
    a = t.cpu().numpy()
    assert (a[n:] == GUARD).all(), "written behind an output"
    return a[:n]


class Pool:
    """Sequences in groups that share their first pages, over shuffled pages; `extra` holders that no table here has."""

    def __init__(self, groups, page, blocks, seed=0, spare=9, extra=0):
        rng = np.random.default_rng(seed)
        self.page, self.blocks = page, blocks
        self.lens = [n for g in groups for n in g]
        need = [ref.pages_of(max(n, 0), page) for n in self.lens]
        self.n_pages = sum(need) + spare
        order = list(rng.permutation(self.n_pages).astype(int))
        self.table = np.full((len(self.lens), blocks), -5, dtype=np.int32)
        b = 0
        for g in groups:
            first = b
            for n in g:
                k = min(need[b], blocks)
                common = 0 if b == first or n <= 0 else int(rng.integers(0, min(self.lens[first], n) // page + 1))
                self.table[b, :common] = self.table[first, :common]
                for j in range(common, k):
                    self.table[b, j] = order.pop()
                b += 1
        self.free = order
        self.held = np.zeros(self.n_pages, dtype=int)
        for b, n in enumerate(need):
            self.held[self.table[b, :min(n, blocks)]] += 1
        kept = np.flatnonzero(self.held)
        self.held[kept[rng.permutation(len(kept))[:extra]]] += 1
        self.shares = np.maximum(self.held - 1, 0)


def fork_ref(p, parents, n_free):
    """One child after the other over holders' counts: lens, table, shares, free, copies."""
    held, free = p.held.copy(), list(p.free[:n_free])
    rows = [p.table[b, :ref.pages_of(n, p.page)] for b, n in enumerate(p.lens)]
    for row in rows:
        held[row] -= 1
    k = len(parents)
    table = np.full((k, p.blocks), GUARD, dtype=np.int32)
    lens, src, dst, count, kept = [0] * k, [-1] * k, [-1] * k, [0] * k, set()
    for i, b in enumerate(parents):
        if not 0 <= b < len(rows):
            continue
        row, lens[i] = rows[b].copy(), p.lens[b]
        if p.lens[b] % p.page and b in kept:
            src[i], count[i] = int(row[-1]), p.lens[b] % p.page
            dst[i] = row[-1] = free.pop()
        kept.add(b)
        table[i, :len(row)] = row
        held[row] += 1
    free += [int(x) for x in np.flatnonzero((p.held > 0) & (held == 0))]
    return lens, table, np.maximum(held - 1, 0), free, src, dst, count


class Fork:
    def __init__(self, pool, parents, n_free=None, in_place=False, ws=None):
        from qwen2_decoder_forward_decode_gb300 import binding
        p = self.p = pool
        self.parents, self.in_place = list(parents), in_place
        self.n_free = len(p.free) if n_free is None else n_free
        k = len(parents)
        self.tlens, self.ttable, self.tparents, self.tshares = dev(p.lens), dev(p.table), dev(self.parents), torch.cat([dev(p.shares), guarded(0)])
        self.tfree = torch.cat([dev(p.free), torch.full((p.n_pages - len(p.free),), -9, dtype=torch.int32, device="cuda"), guarded(0)])
        self.tn = dev([self.n_free])
        self.lens, self.table, self.src, self.dst, self.count = guarded(k), guarded(k * p.blocks), guarded(k), guarded(k), guarded(k)
        self.shares, self.free, self.n = (self.tshares, self.tfree, self.tn) if in_place else (guarded(p.n_pages), guarded(p.n_pages), guarded(1))
        self.ws = torch.zeros(binding.page_fork_workspace(p.n_pages), dtype=torch.uint8, device="cuda") if ws is None else ws
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self):
        from qwen2_decoder_forward_decode_gb300 import binding
        p = self.p
        binding.page_fork(len(p.lens), len(self.parents), p.page, p.n_pages, p.blocks, self.tlens.data_ptr(), self.ttable.data_ptr(), self.tparents.data_ptr(), self.tshares.data_ptr(),
                          self.tfree.data_ptr(), self.tn.data_ptr(), self.lens.data_ptr(), self.table.data_ptr(), self.shares.data_ptr(), self.free.data_ptr(), self.n.data_ptr(),
                          self.src.data_ptr(), self.dst.data_ptr(), self.count.data_ptr(), self.ws.data_ptr(), self.ws.numel(), self.err.data_ptr(), torch.cuda.current_stream().cuda_stream)

    def check(self, err=0):
        torch.cuda.synchronize()
        assert int(self.err) == err
        p, k = self.p, len(self.parents)
        lens, table, shares, free, src, dst, count = fork_ref(p, self.parents, self.n_free)
        assert taken(self.lens, k).tolist() == lens
        np.testing.assert_array_equal(taken(self.table, k * p.blocks).reshape(k, p.blocks), table)
        np.testing.assert_array_equal(taken(self.shares, p.n_pages), shares)
        assert int(self.n[0]) == len(free)
        got = taken(self.free, p.n_pages)
        assert got[:len(free)].tolist() == free
        if not self.in_place:
            assert (got[len(free):] == GUARD).all()
        for a, b in ((self.src, src), (self.dst, dst), (self.count, count)):
            assert taken(a, k).tolist() == b
        ws = self.ws.clone()
        ws[:12] = 0  # what one launch tells the next
        assert not bool(ws.any()), "the workspace is not ready for the next call"


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("groups,page,parents", [
    ([[5]], 4, [0, 0, 0]),                                    # a prompt becomes three samples
    ([[8]], 4, [0, 0, 0]),                                    # its last page is full: nothing to copy
    ([[3]], 16, [0]),
    ([[0], [7]], 4, [0, 0, 1]),                               # an empty sequence has empty children
    ([[9, 9, 9, 9]], 4, [2, 2, 0, 2]),                        # beams, two of which end
    ([[9, 9], [1, 1]], 1, [1, 1, 3, 3]),                      # a page a position
    ([[9, 12, 7], [33]], 8, [-1, 1, -1, 3]),                  # finished sequences
    ([[9, 12, 7], [33]], 8, [-1, -1, -1]),                    # all end
    ([[9, 12, 7], [33]], 8, []),
    ([], 8, [-1, -1]),
    ([[100, 60, 100], [17, 30], [64]], 16, [0, 1, 2, 3, 4, 5]),  # every one goes on
    ([[100, 60, 100], [17, 30], [64]], 16, [5, 4, 3, 2, 1, 0, 0, 5]),
])
def test_fork_matches_the_loop(groups, page, parents, in_place):
    for seed, extra in ((0, 0), (1, 3)):
        f = Fork(Pool(groups, page, 30, seed, extra=extra), parents, in_place=in_place)
        f.run()
        f.check()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("groups,each,hi,page,n_out", [(64, 4, 3000, 16, 4), (300, 8, 200, 7, 8), (4, 1, 60000, 1, 20), (2048, 8, 20, 16, 8), (700, 1, 90, 32, 20)])
def test_large_forks(groups, each, hi, page, n_out, in_place):
    rng = np.random.default_rng(groups)
    lens = [rng.integers(0, hi + 1, each).tolist() for _ in range(groups)]
    pool = Pool(lens, page, ref.pages_of(hi, page) + 1, seed=3, spare=groups * n_out + 5, extra=20)
    parents = (rng.integers(-1, each, (groups, n_out)) + np.arange(groups)[:, None] * each)
    parents[parents < np.arange(groups)[:, None] * each] = -1
    f = Fork(pool, parents.reshape(-1).tolist(), in_place=in_place)
    f.run()
    f.check()


def test_the_most_sequences():
    pool = Pool([[3]] * 16384, 4, 1, spare=40000)
    f = Fork(pool, [b // 2 for b in range(16384)])
    f.run()
    f.check()


@pytest.mark.parametrize("case", ["pages", "length", "long", "count", "negative"])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_fork_that_does_not_fit_changes_nothing(case, in_place):
    pool = Pool([[9, 5], [6]], 4, 4)
    if case == "length":
        pool.lens[1] = -1
    if case == "long":
        pool.lens[1] = 17
    f = Fork(pool, [0, 0, 0, 1, 2, 2], n_free={"pages": 2, "count": pool.n_pages + 1, "negative": -1}.get(case), in_place=in_place)
    shares, free = f.tshares.clone(), f.tfree.clone()
    f.run()
    torch.cuda.synchronize()
    assert int(f.err) == 64
    assert taken(f.lens, 6).tolist() == [0] * 6 and (f.table == GUARD).all()
    assert taken(f.src, 6).tolist() == [-1] * 6 and taken(f.dst, 6).tolist() == [-1] * 6 and taken(f.count, 6).tolist() == [0] * 6
    assert torch.equal(f.shares[:pool.n_pages], shares[:pool.n_pages]) and int(f.n[0]) == f.n_free
    if 0 <= f.n_free <= pool.n_pages:
        assert torch.equal(f.free[:f.n_free], free[:f.n_free])
    # the call after it finds the workspace ready
    good = Pool([[9, 5], [6]], 4, 4)
    f2 = Fork(good, [0, 0, 2], ws=f.ws)
    f2.run()
    f2.check()


def test_bad_parents_and_pages_are_reported():
    pool = Pool([[9, 5], [6]], 4, 4)
    f = Fork(pool, [0, 7, -2, 2])
    f.run()
    f.check(err=32)
    pool = Pool([[9, 9]], 4, 4)
    pool.table[0, 1] = pool.n_pages
    pool.table[1, 0] = -3
    f = Fork(pool, [0, 0])
    f.run()
    torch.cuda.synchronize()
    assert int(f.err) == 32
    assert taken(f.table, 8).reshape(2, 4)[0, 1] == pool.n_pages  # as it was


@pytest.mark.parametrize("in_place", [False, True])
def test_negative_counts_are_zeros(in_place):
    pool = Pool([[60, 50], [33], [20, 20]], 4, 16)
    f = Fork(pool, [0, 0, 0, 2, 2, 2, 2, 1, 3], in_place=in_place)
    f.tshares[:pool.n_pages] = torch.where(f.tshares[:pool.n_pages] == 0, torch.full_like(f.tshares[:pool.n_pages], -3), f.tshares[:pool.n_pages])
    f.run()
    if in_place:  # (counts that nobody touched stay as they were)
        f.shares[:pool.n_pages].clamp_(min=0)
    f.check()


def test_a_captured_fork_follows_the_device():
    """Two forks one after the other as a graph, there and back, with other parents at each replay."""
    from qwen2_decoder_forward_decode_gb300 import binding
    rng = np.random.default_rng(5)
    pool = Pool([[200, 180, 220, 150]] * 3, 16, 20, spare=60)
    f = Fork(pool, list(range(12)), in_place=True)
    back = dev(np.arange(12))

    def twice():
        f.run()
        p = f.p
        binding.page_fork(12, 12, p.page, p.n_pages, p.blocks, f.lens.data_ptr(), f.table.data_ptr(), back.data_ptr(), f.shares.data_ptr(), f.free.data_ptr(), f.n.data_ptr(), f.tlens.data_ptr(),
                          f.ttable.data_ptr(), f.shares.data_ptr(), f.free.data_ptr(), f.n.data_ptr(), f.src.data_ptr(), f.dst.data_ptr(), f.count.data_ptr(), f.ws.data_ptr(), f.ws.numel(),
                          f.err.data_ptr(), torch.cuda.current_stream().cuda_stream)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        twice()
    lens, table, held, free = list(pool.lens), pool.table.copy(), pool.held.copy(), list(pool.free)
    for _ in range(6):
        parents = (rng.integers(0, 4, (3, 4)) + np.arange(3)[:, None] * 4).reshape(-1).tolist()
        f.tparents.copy_(dev(parents))
        g.replay()
        torch.cuda.synchronize()
        assert int(f.err) == 0
        state = Pool([[]], 16, 20)
        state.lens, state.table, state.held, state.free = lens, table, held, free
        lens, new, shares, free, *_ = fork_ref(state, parents, len(free))
        table = np.where(new == GUARD, table, new)
        held = np.where(np.isin(np.arange(pool.n_pages), [x for b in range(12) for x in table[b, :ref.pages_of(lens[b], 16)]]), shares + 1, 0)
        assert f.tlens.tolist() == lens
        for b in range(12):
            k = ref.pages_of(lens[b], 16)
            assert f.ttable[b, :k].tolist() == table[b, :k].tolist()
        np.testing.assert_array_equal(taken(f.shares, pool.n_pages), shares)
        assert f.free[:int(f.n)].tolist() == free
    assert sorted(free + [int(x) for x in np.flatnonzero(held)]) == list(range(pool.n_pages))


# ---- copies ------------------------------------------------------------------------------------------


def caches(layers, n_pages, nkv, page, hd, dtype, layout, gap=0, seed=0):
    """Views into larger buffers, gap * 16 bytes between rows, and the array for the call."""
    from qwen2_decoder_forward_decode_gb300 import binding
    unit = {"f32": 4, "f16": 8, "bf16": 8}[dtype]
    gen = torch.Generator("cuda").manual_seed(seed)
    shape = (n_pages, nkv, page, hd + gap * unit) if layout == "head" else (n_pages, page, nkv, hd + gap * unit)
    whole = [[torch.randn(shape, device="cuda", generator=gen).to(ref.torch_dtype(dtype)) for _ in range(2)] for _ in range(layers)]
    st = whole[0][0].stride()
    head, pos = (st[1], st[2]) if layout == "head" else (st[2], st[1])
    return whole, binding.paged_kv_array([binding.PagedKV(k.data_ptr(), v.data_ptr(), ref.CODE[dtype], n_pages, page, nkv, hd, st[0], head, pos) for k, v in whole])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layers,n,nkv,page,hd,layout,gap,filled", [
    (1, 1, 1, 1, 8, "head", 0, False), (2, 5, 2, 16, 128, "head", 0, True), (28, 16, 2, 16, 128, "head", 0, True), (3, 40, 3, 7, 80, "position", 1, True),
    (1, 300, 4, 64, 128, "position", 0, False), (128, 3, 1, 5, 16, "head", 2, True), (2, 9, 4, 256, 256, "head", 0, False),
])
def test_copies_match_the_loop(dtype, layers, n, nkv, page, hd, layout, gap, filled):
    from qwen2_decoder_forward_decode_gb300 import binding
    rng = np.random.default_rng(n)
    n_pages = 2 * n + 3
    whole, kvs = caches(layers, n_pages, nkv, page, hd, dtype, layout, gap)
    want = [[t.clone() for t in pair] for pair in whole]
    order = rng.permutation(n_pages)
    src, dst, count = order[:n].copy(), order[n:2 * n], rng.integers(0, page + 1, n) if filled else np.full(n, page)
    if n > 4:
        src[::4] = -1
    for pair in want:
        for t in pair:
            rows = (t.transpose(1, 2) if layout == "head" else t)[..., :hd]
            for a, b, m in zip(src.tolist(), dst.tolist(), count.tolist()):
                if a >= 0:
                    rows[b, :m] = rows[a, :m]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tsrc, tdst, tcount = dev(src), dev(dst), dev(count)
    binding.page_copy(kvs, layers, n, tsrc.data_ptr(), tdst.data_ptr(), tcount.data_ptr() if filled else None, err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert int(err) == 0
    for a, b in zip(whole, want):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_bad_copies_are_left_out_and_reported():
    from qwen2_decoder_forward_decode_gb300 import binding
    whole, kvs = caches(2, 8, 2, 16, 64, "f16", "head")
    want = [[t.clone() for t in pair] for pair in whole]
    for src, dst, count in ((8, 1, 3), (-2, 1, 3), (0, 8, 3), (0, -1, 3), (0, 1, 17), (0, 1, -1)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        a, b, m = dev([src, 2]), dev([dst, 3]), dev([count, 16])
        binding.page_copy(kvs, 2, 2, a.data_ptr(), b.data_ptr(), m.data_ptr(), err.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert int(err) == 32
        for pair in want:
            for t in pair:
                t[3] = t[2]
        assert all(torch.equal(x, y) for p, q in zip(whole, want) for x, y in zip(p, q))


@pytest.mark.parametrize("dtype", ["f16"])
def test_copies_beyond_32_bits(dtype):
    """A cache of 5 G elements: the pages' offsets pass 2^32."""
    from qwen2_decoder_forward_decode_gb300 import binding
    page, nkv, hd = 64, 4, 128
    n_pages = 5 * 2 ** 30 // (page * nkv * hd)
    k = torch.zeros(n_pages, page, nkv, hd, dtype=torch.float16, device="cuda")
    k[n_pages - 1].normal_()
    k[3].normal_()
    want = k[n_pages - 1].clone(), k[3].clone()
    kvs = binding.paged_kv_array([binding.PagedKV(k.data_ptr(), k.data_ptr(), 2, n_pages, page, nkv, hd, page * nkv * hd, hd, nkv * hd)])
    err, src, dst = torch.zeros(1, dtype=torch.int32, device="cuda"), dev([n_pages - 1, 3]), dev([5, n_pages - 2])
    binding.page_copy(kvs, 1, 2, src.data_ptr(), dst.data_ptr(), None, err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(k[5], want[0]) and torch.equal(k[n_pages - 2], want[1])


# ---- compaction --------------------------------------------------------------------------------------


class Compact:
    def __init__(self, n_pages, needs, page, blocks, max_moves, seed=0, in_place=False, shares=True, ws=None):
        from qwen2_decoder_forward_decode_gb300 import binding
        rng = np.random.default_rng(seed)
        self.n_pages, self.page, self.blocks, self.max_moves, self.in_place = n_pages, page, blocks, max_moves, in_place
        order = rng.permutation(n_pages)
        self.table = np.full((len(needs), blocks), -5, dtype=np.int32)
        at = 0
        for b, k in enumerate(needs):
            self.table[b, :k] = order[at:at + k]
            at += k
            if shares and b % 3 == 1:
                c = min(k, needs[b - 1]) // 2
                self.table[b, :c] = self.table[b - 1, :c]
        self.lens = [max(0, k * page - int(rng.integers(0, page))) for k in needs]
        held = np.zeros(n_pages, dtype=int)
        for b, k in enumerate(needs):
            held[self.table[b, :k]] += 1
        self.shares = np.maximum(held - 1, 0)
        self.free = rng.permutation(np.flatnonzero(held == 0)).tolist()
        self.tlens, self.ttable, self.tshares = dev(self.lens), torch.cat([dev(self.table).reshape(-1), guarded(0)]), torch.cat([dev(self.shares), guarded(0)])
        self.tfree, self.tn = torch.cat([dev(self.free + [-9] * (n_pages - len(self.free))), guarded(0)]), dev([len(self.free)])
        self.otable, self.oshares, self.ofree = (self.ttable, self.tshares, self.tfree) if in_place else (guarded(self.table.size), guarded(n_pages), guarded(n_pages))
        self.src, self.dst, self.n = guarded(max_moves), guarded(max_moves), guarded(1)
        self.with_shares = shares
        self.ws = torch.zeros(binding.page_compact_workspace(n_pages), dtype=torch.uint8, device="cuda") if ws is None else ws
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self):
        from qwen2_decoder_forward_decode_gb300 import binding
        s = self.with_shares
        binding.page_compact(len(self.lens), self.page, self.n_pages, self.blocks, self.max_moves, self.tlens.data_ptr(), self.ttable.data_ptr(), self.tshares.data_ptr() if s else None,
                             self.tfree.data_ptr(), self.tn.data_ptr(), self.otable.data_ptr(), self.oshares.data_ptr() if s else None, self.ofree.data_ptr(), self.src.data_ptr(),
                             self.dst.data_ptr(), self.n.data_ptr(), self.ws.data_ptr(), self.ws.numel(), self.err.data_ptr(), torch.cuda.current_stream().cuda_stream)

    def check(self):
        torch.cuda.synchronize()
        assert int(self.err) == 0
        free, n_free = set(self.free), len(self.free)
        live = self.n_pages - n_free
        pairs = list(zip([p for p in range(self.n_pages - 1, live - 1, -1) if p not in free], sorted(p for p in free if p < live)))[:self.max_moves]
        to, shares = np.arange(self.n_pages), self.shares.copy()
        for a, b in pairs:
            to[a], shares[b], shares[a] = b, self.shares[a], 0
            free.remove(b)
            free.add(a)
        table = self.table.copy()
        for b, length in enumerate(self.lens):
            k = ref.pages_of(length, self.page)
            table[b, :k] = to[table[b, :k]]
        assert int(self.n[0]) == len(pairs)
        rest = [-1] * (self.max_moves - len(pairs))
        assert taken(self.src, self.max_moves).tolist() == [a for a, _ in pairs] + rest
        assert taken(self.dst, self.max_moves).tolist() == [b for _, b in pairs] + rest
        np.testing.assert_array_equal(taken(self.otable, table.size).reshape(table.shape), table)
        assert taken(self.ofree, self.n_pages)[:n_free].tolist() == sorted(free, reverse=True)
        if self.with_shares:
            np.testing.assert_array_equal(taken(self.oshares, self.n_pages), shares)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_pages,needs,page,moves", [
    (1, [], 4, 3), (1, [1], 4, 3), (5, [2, 1], 4, 9), (40, [3, 0, 7, 1], 16, 40), (40, [3, 0, 7, 1], 16, 2), (40, [3, 0, 7, 1], 16, 0), (64, [64], 1, 10), (64, [], 1, 10),
    (2047, [300, 17, 500], 7, 1000), (2048, [300, 17, 500], 7, 100), (2049, [1] * 700, 16, 2049), (10000, [40] * 100, 16, 10000), (70001, [9] * 5000, 16, 30000), (70001, [9] * 5000, 16, 333),
])
def test_compaction_matches_the_loop(n_pages, needs, page, moves, in_place):
    c = Compact(n_pages, needs, page, max(needs + [1]) + 1, moves, in_place=in_place)
    c.run()
    c.check()
    if not in_place:  # the workspace is ready for the next call
        c.run()
        c.check()


def test_a_pool_of_many_ranges():
    rng = np.random.default_rng(1)
    c = Compact(2200000, rng.integers(0, 1200, 2000).tolist(), 16, 1200, 400000)
    c.run()
    c.check()


def test_compaction_without_counts_and_twice():
    c = Compact(500, [40, 60, 3], 4, 70, 500, shares=False)
    c.run()
    c.check()
    c.run()
    c.check()


@pytest.mark.parametrize("case", ["twice", "outside", "below", "count", "length"])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_bad_pool_is_left_as_it_is(case, in_place):
    c = Compact(100, [20, 30], 4, 40, 50, in_place=in_place)
    if case == "twice":
        c.tfree[3] = c.tfree[4]
    if case == "outside":
        c.tfree[3] = 100
    if case == "below":
        c.tfree[3] = -1
    if case == "count":
        c.tn.fill_(101)
    if case == "length":
        c.tlens[1] = 161
    table, shares, free = c.ttable.clone(), c.tshares.clone(), c.tfree.clone()
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == (64 if case in ("count", "length") else 32)
    assert torch.equal(c.otable, table) and torch.equal(c.oshares, shares) and int(c.n[0]) == 0
    n = min(int(c.tn), 100)
    assert torch.equal(c.ofree[:n], free[:n])
    assert taken(c.src, 50).tolist() == [-1] * 50 and taken(c.dst, 50).tolist() == [-1] * 50
    good = Compact(100, [20, 30], 4, 40, 50, seed=2, ws=c.ws)
    good.run()
    good.check()


def test_a_bad_table_entry_stays():
    c = Compact(100, [20, 30], 4, 40, 50)
    c.ttable[5] = 100
    c.ttable[40 + 7] = -2
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == 32 and int(c.otable[5]) == 100 and int(c.otable[47]) == -2


def test_forks_and_compactions_on_two_streams():
    """Calls at the same time with workspaces of their own."""
    pools = [Pool([[300, 280, 310, 299]] * 20, 16, 24, seed=i, spare=100) for i in range(2)]
    parents = [0, 0, 1, 3] * 20
    forks = [Fork(p, [x + 4 * (i // 4) for i, x in enumerate(parents)]) for p in pools]
    packs = [Compact(5000, [40] * 60, 16, 41, 5000, seed=i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, f, c in zip(streams, forks, packs):
            with torch.cuda.stream(s):
                f.run()
                c.run()
    torch.cuda.synchronize()
    for f, c in zip(forks, packs):
        f.check()
        c.check()
