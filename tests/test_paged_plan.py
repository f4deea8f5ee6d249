"""Page plans and page release on the GPU against a loop over the sequences: whole numbers, so equal."""
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


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def guarded(n, dtype=torch.int32):
    return torch.full((n + 3,), GUARD, dtype=dtype, device="cuda")


class Plan:
    def __init__(self, lens, new, page, blocks, max_tokens, spare=5, seed=0, n_free=None, in_place=False, null_new=False):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.page, self.blocks, self.max_tokens = list(lens), list(new), page, blocks, max_tokens
        have = [ref.pages_of(max(n, 0), page) for n in lens]
        take = sum(ref.pages_of(max(a + b, 0), page) - h for a, b, h in zip(lens, new, have))
        self.n_pages = sum(have) + max(take, 0) + spare
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(lens), blocks), -5, dtype=np.int32)
        at = 0
        for b, h in enumerate(have):
            h = min(h, blocks)
            self.table[b, :h] = order[at:at + h]
            at += h
        self.free = list(order[at:])
        self.n_free = len(self.free) if n_free is None else n_free
        self.tfree = dev(np.concatenate([self.free, np.full(self.n_pages - len(self.free), -9)]))
        n = len(lens)
        self.tlens, self.tnew = dev(self.lens), None if null_new else dev(self.new)
        self.tn_free = dev([self.n_free])
        self.ttable = torch.cat([dev(self.table).reshape(-1), guarded(0)])
        self.lens_out = torch.cat([self.tlens, guarded(0)]) if in_place else guarded(n)
        if in_place:
            self.tlens = self.lens_out
        self.n_free_out = self.tn_free if in_place else guarded(1)
        self.cu, self.positions, self.slots = guarded(n + 1), guarded(max_tokens), guarded(max_tokens, torch.int64)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self):
        from qwen2_decoder_forward_decode_gb300 import binding
        binding.page_plan(len(self.lens), self.page, self.n_pages, self.blocks, self.max_tokens, self.tlens.data_ptr(), None if self.tnew is None else self.tnew.data_ptr(),
                          self.tfree.data_ptr(), self.tn_free.data_ptr(), self.ttable.data_ptr(), self.lens_out.data_ptr(), self.n_free_out.data_ptr(), self.cu.data_ptr(),
                          self.positions.data_ptr(), self.slots.data_ptr(), self.err.data_ptr(), torch.cuda.current_stream().cuda_stream)

    def got(self):
        torch.cuda.synchronize()
        n = len(self.lens)
        out = []
        for t, size in ((self.ttable, n * self.blocks), (self.lens_out, n), (self.cu, n + 1), (self.positions, self.max_tokens), (self.slots, self.max_tokens)):
            a = t.cpu().numpy()
            assert (a[size:] == GUARD).all(), "written behind an output"
            out.append(a[:size])
        return [out[0].reshape(n, self.blocks)] + out[1:] + [int(self.n_free_out[0]), int(self.err)]

    def check(self):
        table, lens, cu, positions, slots, n_free, err = self.got()
        w = ref.plan(self.lens, self.new, self.page, self.table, self.free, self.max_tokens)
        for a, b in zip((table, lens, cu, positions, slots), (w[0], w[1], w[3], w[4], w[5])):
            np.testing.assert_array_equal(a, b)
        assert (n_free, err) == (len(w[2]), 0)
        free = self.tfree.cpu().numpy()
        np.testing.assert_array_equal(free[:len(self.free)], self.free)


@pytest.mark.parametrize("n,page,hi,new_hi,pad,in_place,null_new", [
    (1, 16, 0, 1, 0, False, False),        # the first token of one sequence
    (1, 1, 5, 3, 2, True, False),          # a page a position
    (5, 7, 40, 30, 9, False, False),
    (31, 16, 100, 1, 0, True, True),       # a decode step, updated in place
    (200, 16, 300, 70, 100, False, False),
    (512, 16, 3000, 1, 0, False, True),
    (1025, 32, 500, 5, 33, True, False),   # one more than a block of threads
    (64, 16, 100, 2500, 50, False, False),  # prefill
    (7, 128, 1000, 9000, 1, True, False),
    (16384, 16, 20, 2, 0, False, False),   # the most sequences
])
def test_plan_matches_the_loop(n, page, hi, new_hi, pad, in_place, null_new):
    rng = np.random.default_rng(n + page)
    lens = rng.integers(0, hi + 1, n)
    new = np.ones(n, dtype=np.int64) if null_new else rng.integers(0, new_hi + 1, n)
    blocks = max(1, max(ref.pages_of(a + b, page) for a, b in zip(lens, new))) + 1
    p = Plan(lens.tolist(), new.tolist(), page, blocks, int(new.sum()) + pad, in_place=in_place, null_new=null_new)
    p.run()
    p.check()


def test_every_sequence_idle():
    p = Plan([3, 0, 16], [0, 0, 0], 16, 4, 10)
    p.run()
    p.check()


def test_no_sequence_and_no_token():
    p = Plan([], [], 16, 1, 6)
    p.run()
    table, lens, cu, positions, slots, n_free, err = p.got()
    assert cu.tolist() == [0] and positions.tolist() == [0] * 6 and slots.tolist() == [-1] * 6 and n_free == p.n_free and err == 0
    p = Plan([4, 9], [0, 0], 16, 1, 0)
    p.run()
    p.check()


@pytest.mark.parametrize("over", [
    dict(lens=[3, 16], new=[1, 1], n_free=0),                        # no page left for the second
    dict(lens=[3, 16], new=[4, 5], max_tokens=8),                    # too many tokens
    dict(lens=[3, 60], new=[1, 5]),                                  # beyond the table's row
    dict(lens=[3, -1], new=[1, 1]), dict(lens=[3, 4], new=[1, -1]),  # no lengths
    dict(lens=[3, 4], new=[1, 1], n_free=-1), dict(lens=[3, 4], new=[1, 1], n_free=10 ** 6),
    dict(lens=[3, 2 ** 31 - 1], new=[1, 2 ** 31 - 1]),               # sums beyond 32 bits
])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_step_that_does_not_fit_changes_nothing(over, in_place):
    from qwen2_decoder_forward_decode_gb300 import binding
    o = dict(over)
    big = o["lens"][1] > 2 ** 30
    p = Plan([o["lens"][0], 4] if big else o["lens"], [1, 1] if big else o["new"], 16, 4, o.get("max_tokens", 64), n_free=o.get("n_free"), in_place=in_place)
    if big:
        p.lens, p.new = o["lens"], o["new"]
        p.tlens[:2] = torch.tensor(o["lens"], dtype=torch.int32)
        p.tnew = dev(o["new"])
    p.run()
    table, lens, cu, positions, slots, n_free, err = p.got()
    assert err == binding.DEV_CAPACITY
    np.testing.assert_array_equal(table, p.table)
    assert lens.tolist() == p.lens and n_free == p.n_free
    assert (cu == 0).all() and (positions == 0).all() and (slots == -1).all()


def test_bad_page_ids_give_no_slot():
    from qwen2_decoder_forward_decode_gb300 import binding
    p = Plan([3, 16, 5], [2, 2, 1], 16, 4, 6)
    p.ttable[0] = p.n_pages                 # the page that sequence 0 goes on filling
    p.tfree[p.n_free - 1] = -1              # the page that sequence 1 takes
    p.run()
    table, lens, cu, positions, slots, n_free, err = p.got()
    assert err == binding.DEV_PAGE
    assert slots[:4].tolist() == [-1] * 4 and slots[4] == int(p.table[2, 0]) * 16 + 5 and slots[5] == -1
    assert table[1, 1] == -1 and lens.tolist() == [5, 18, 6] and n_free == p.n_free - 1


def test_a_captured_plan_follows_the_device_lengths():
    """A decode loop as a graph: lengths and the free count advance in place at every replay."""
    p = Plan([0, 14, 31, 7], [1] * 4, 16, 8, 4, spare=40, in_place=True, null_new=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.run()
    side.synchronize()
    p.check()
    lens, free, table = [n + 1 for n in p.lens], p.free[:int(p.n_free_out[0])], p.got()[0].copy()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for _ in range(20):
        g.replay()
        p.lens, p.free, p.table = lens, free, table
        p.check()
        table, lens, free = ref.plan(lens, p.new, 16, table, free, 4)[:3]


def release_want(lens, done, page, table, free, n_pages):
    free = list(free)
    for b, d in enumerate(done):
        if d:
            free += table[b, :ref.pages_of(lens[b], page)].tolist()
    return free, [0 if d else n for n, d in zip(lens, done)]


def release(p, done, in_place=False):
    from qwen2_decoder_forward_decode_gb300 import binding
    binding.page_release(len(p.lens), p.page, p.n_pages, p.blocks, p.tlens.data_ptr(), dev(done).data_ptr(), p.ttable.data_ptr(), p.tfree.data_ptr(), p.tn_free.data_ptr(),
                         p.lens_out.data_ptr(), p.n_free_out.data_ptr(), p.err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()


@pytest.mark.parametrize("n,page,hi,in_place", [(1, 16, 1, False), (6, 7, 50, True), (300, 16, 400, False), (1500, 1, 20, True), (16384, 16, 40, False)])
def test_release_matches_the_loop(n, page, hi, in_place):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, hi + 1, n).tolist()
    p = Plan(lens, [0] * n, page, max(1, max(ref.pages_of(x, page) for x in lens)) + 1, 0, in_place=in_place)
    done = rng.integers(0, 2, n) * rng.integers(1, 5, n)
    before = p.tfree.cpu().numpy()
    release(p, done)
    free, left = release_want(lens, done, page, p.table, p.free, p.n_pages)
    assert int(p.n_free_out[0]) == len(free) and int(p.err) == 0
    got = p.tfree.cpu().numpy()
    np.testing.assert_array_equal(got[:len(free)], free)
    np.testing.assert_array_equal(got[len(free):], before[len(free):])
    np.testing.assert_array_equal(p.lens_out.cpu().numpy(), left + [GUARD] * 3)
    np.testing.assert_array_equal(p.ttable.cpu().numpy()[:-3].reshape(p.table.shape), p.table)


@pytest.mark.parametrize("case", ["list full", "negative", "beyond the table", "bad count"])
def test_a_release_that_does_not_fit_changes_nothing(case):
    from qwen2_decoder_forward_decode_gb300 import binding
    p = Plan([20, 30], [0, 0], 16, 4, 0)
    if case == "list full":
        p.tn_free[0] = p.n_pages - 3
    if case == "bad count":
        p.tn_free[0] = p.n_pages + 1
    if case == "negative":
        p.tlens[1] = -4
    if case == "beyond the table":
        p.tlens[1] = 65
    free, lens, count = p.tfree.clone(), p.tlens.clone(), int(p.tn_free[0])
    release(p, [1, 1])
    assert int(p.err) == binding.DEV_CAPACITY and int(p.n_free_out[0]) == count
    assert torch.equal(p.tfree, free) and torch.equal(p.lens_out[:2], lens)


def test_a_bad_page_id_is_released_and_reported():
    from qwen2_decoder_forward_decode_gb300 import binding
    p = Plan([20, 30], [0, 0], 16, 4, 0)
    p.ttable[1] = 10 ** 6
    release(p, [1, 0])
    assert int(p.err) == binding.DEV_PAGE
    assert p.tfree[len(p.free):len(p.free) + 2].tolist() == [int(p.table[0, 0]), 10 ** 6]


def test_host_memory_is_refused():
    from qwen2_decoder_forward_decode_gb300 import binding
    p = Plan([20, 30], [0, 0], 16, 4, 0)
    p.tlens = p.tlens.cpu()
    with pytest.raises(binding.QwError) as e:
        p.run()
    assert e.value.status == 1 and "device memory" in str(e.value)


def test_batches_of_many_sizes_from_several_threads():
    """The kernels' shared memory grows with the number of sequences: calls of other sizes in other host threads must not
    change what a launch is allowed."""
    import threading
    from qwen2_decoder_forward_decode_gb300 import binding
    L = binding.lib()
    plans = [Plan([5] * n, [0] * (n - 9) + [1] * 9, 16, 1, 9) for n in (16384, 6000, 16384, 6000, 9000)]
    streams, done = [torch.cuda.Stream() for _ in plans], dev([0] * 16384)
    torch.cuda.synchronize()
    failed = []

    def loop(p, stream):
        ptr = lambda *names: [getattr(p, n).data_ptr() for n in names]  # noqa: E731
        plan = [len(p.lens), p.page, p.n_pages, p.blocks, p.max_tokens] + ptr("tlens", "tnew", "tfree", "tn_free", "ttable", "lens_out", "n_free_out", "cu", "positions", "slots", "err")
        other = torch.zeros(len(p.lens) + 1, dtype=torch.int32, device="cuda")
        back = [len(p.lens), p.page, p.n_pages, p.blocks] + ptr("tlens") + [done.data_ptr()] + ptr("ttable", "tfree", "tn_free") + [other.data_ptr(), other.data_ptr() + 4 * len(p.lens)] + ptr("err")
        for _ in range(5000):  # (prepared calls: the more of a thread's time is in the library, the nearer they come)
            if L.qw_op_page_plan(*plan, stream.cuda_stream) or L.qw_op_page_release(*back, stream.cuda_stream):
                failed.append((len(p.lens), L.qw_last_error()))

    threads = [threading.Thread(target=loop, args=a) for a in zip(plans, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, (len(failed), failed[0])
    for p in plans:
        p.check()


@pytest.mark.parametrize("in_place", [False, True])
def test_lengths_end_at_31_bits(in_place):
    """Tables whose rows hold more positions than a length can count: the last length fits, the next does not."""
    from qwen2_decoder_forward_decode_gb300 import binding
    p = Plan([2 ** 31 - 2, 5], [1, 1], 2 ** 20, 4096, 8, in_place=in_place)
    p.run()
    p.check()
    assert int(p.lens_out[0]) == 2 ** 31 - 1
    for lens, new in (([2 ** 31 - 1, 5], [1, 1]), ([2 ** 31 - 2, 5], [2, 1]), ([5, 2 ** 30], [1, 2 ** 30])):
        p = Plan(lens, new, 2 ** 20, 4096, 8, in_place=in_place)
        p.run()
        table, lens_out, cu, positions, slots, n_free, err = p.got()
        assert err == binding.DEV_CAPACITY
        np.testing.assert_array_equal(table, p.table)
        assert lens_out.tolist() == lens and n_free == p.n_free
        assert (cu == 0).all() and (positions == 0).all() and (slots == -1).all()


def test_large_steps_in_place_captured():
    """Steps that take all SMs and update the lengths and the free count in place, as one graph: plan, then release."""
    from qwen2_decoder_forward_decode_gb300 import binding
    rng = np.random.default_rng(1)
    lens, new = rng.integers(0, 3000, 60).tolist(), rng.integers(100, 700, 60).tolist()
    p = Plan(lens, new, 1, max(a + b for a, b in zip(lens, new)), sum(new) + 50, in_place=True)
    assert p.max_tokens > 8192 and p.n_pages > 8192
    done = rng.integers(0, 2, 60).tolist()
    tdone = dev(done)
    kept = [(t, t.clone()) for t in (p.tlens, p.tn_free, p.ttable, p.tfree)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
        s = torch.cuda.current_stream().cuda_stream
        lens_mid, free_mid = p.tlens.clone(), p.tn_free.clone()
        binding.page_release(60, p.page, p.n_pages, p.blocks, p.tlens.data_ptr(), tdone.data_ptr(), p.ttable.data_ptr(), p.tfree.data_ptr(), p.tn_free.data_ptr(), p.tlens.data_ptr(),
                             p.tn_free.data_ptr(), p.err.data_ptr(), s)
    table, lens2, free, cu, positions, slots = ref.plan(lens, new, p.page, p.table, p.free, p.max_tokens)
    back, left = release_want(lens2, done, p.page, table, free, p.n_pages)
    for _ in range(3):
        for t, was in kept:
            t.copy_(was)
        g.replay()
        got = p.got()
        for a, b in zip((got[0], got[2], got[3], got[4]), (table, cu, positions, slots)):
            np.testing.assert_array_equal(a, b)
        assert lens_mid[:60].tolist() == lens2 and int(free_mid) == len(free)
        assert got[1].tolist() == left and got[5:] == [len(back), 0]
        np.testing.assert_array_equal(p.tfree.cpu().numpy()[:len(back)], back)
