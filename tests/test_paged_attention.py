"""Decode attention over a paged cache against the softmax formula in 64 bits."""
import math

import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
TYPES = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Call:
    def __init__(self, lens, nq, nkv, hd, page, io, cache, layout="head", seed=0, q_scale=2.0, pad=0, scale=None, **kw):
        from qwen2_decoder_forward_decode_gb300 import binding
        rng = np.random.default_rng(seed + len(lens) + hd)
        self.nq, self.nkv, self.hd, self.io = nq, nkv, hd, io
        self.c = ref.PagedCache(rng, lens, nkv, hd, page, cache, layout, **kw)
        n = len(lens)
        q = torch.from_numpy(q_scale * rng.standard_normal((n, nq, hd))).to(ref.torch_dtype(io))
        self.q = q.double().numpy()
        self.tq = torch.full((n + 1, nq * hd + pad), float("nan"), dtype=q.dtype)  # (one more row than sequences)
        self.tq[:n, :nq * hd] = q.reshape(n, -1)
        self.tq = self.tq.cuda()
        self.out = torch.full_like(self.tq, 3.0)
        self.lse = torch.full((n + 1, nq), 3.0, device="cuda")
        self.scale = 1 / math.sqrt(hd) if scale is None else scale
        self.ws = torch.zeros(binding.paged_attention_workspace(nq, nkv, hd), dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, out=None, lse=True):
        from qwen2_decoder_forward_decode_gb300 import binding
        out = self.out if out is None else out
        binding.paged_attention(self.c.kv, len(self.c.lens), self.nq, self.c.ttable.data_ptr(), self.c.blocks, self.c.tlens.data_ptr(), ref.CODE[self.io], self.tq.data_ptr(), self.tq.shape[1],
                                self.scale, out.data_ptr(), out.shape[1], self.lse.data_ptr() if lse else None, self.ws.data_ptr(), self.ws.numel(), self.err.data_ptr(),
                                torch.cuda.current_stream().cuda_stream)

    def check(self, out=None, err=0, lse=True, kv=None):
        torch.cuda.synchronize()
        out = self.out if out is None else out
        assert int(self.err) == err
        n, g, width = len(self.c.lens), self.nq // self.nkv, self.nq * self.hd
        got = out.double().cpu().numpy()
        if out is self.out:
            assert (got[n:] == 3.0).all() and (got[:, width:] == 3.0).all(), "written outside the rows"
        got, tl = got[:n, :width].reshape(n, self.nq, self.hd), self.lse.double().cpu().numpy()
        assert (tl[n:] == 3.0).all()
        for b in range(n):
            for h in range(self.nkv):
                k, v = (self.c.k[b][:, h], self.c.v[b][:, h]) if kv is None else kv(b, h)
                heads = slice(h * g, (h + 1) * g)
                o, l, bound = ref.attention(self.q[b, heads], k, v, self.scale)
                tol = bound + (ref.EPS_HALF[self.io] if self.io != "f32" else 0) * (np.abs(o) + bound) + ref.TINY[self.io]
                np.testing.assert_array_less(np.abs(got[b, heads] - o), tol + 1e-30, err_msg=f"sequence {b} KV head {h} length {self.c.lens[b]}")
                if lse:
                    # the scores' bound, a rounded sum of exponentials, and one step of the result
                    ds = (8 * math.sqrt(self.hd) + 4) * ref.U * abs(self.scale) * (np.abs(self.q[b, heads]) @ np.abs(k).T).max(initial=0)
                    with np.errstate(invalid="ignore"):
                        off = np.where(l == tl[b, heads], 0.0, np.abs(tl[b, heads] - l))
                    assert np.all(off <= ds + (8 * math.sqrt(len(k)) + 8) * ref.U + ref.U * np.where(np.isfinite(l), np.abs(l), 0)), (b, h)


@pytest.mark.parametrize("io,cache", TYPES)
@pytest.mark.parametrize("nq,nkv,hd", [(12, 2, 128), (14, 2, 64), (4, 4, 16), (28, 4, 128), (3, 1, 32), (16, 1, 96), (9, 3, 80), (20, 1, 64), (40, 2, 128), (2, 1, 256), (1, 1, 8)])
@pytest.mark.parametrize("page,layout", [(16, "head"), (7, "position")])
def test_ragged_lengths(io, cache, nq, nkv, hd, page, layout):
    c = Call([0, 1, 2, 15, 16, 17, 63, 64, 65, 0, 100, 129, 300], nq, nkv, hd, page, io, cache, layout)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache", TYPES)
@pytest.mark.parametrize("lens,page", [([2000], 16), ([1], 1), ([5000, 3], 64), ([777] * 9, 256), ([31, 4000, 0, 64, 1], 128), ([1500, 1499], 1)])
def test_long_and_lone_sequences(io, cache, lens, page):
    c = Call(lens, 12, 2, 128, page, io, cache)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 64), ("bf16", "bf16", 128), ("f32", "f32", 32)])
def test_many_sequences(io, cache, hd):
    """More sequences than a block has threads, most of them short."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 70, 700)
    lens[rng.integers(0, 700, 30)] = rng.integers(100, 600, 30)
    c = Call(lens.tolist(), 4, 2, hd, 16, io, cache)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache", TYPES)
def test_very_long_context(io, cache):
    c = Call([70001], 4, 1, 64, 16, io, cache)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache", TYPES)
def test_strides_gaps_and_no_lse(io, cache):
    c = Call([40, 3, 129], 6, 2, 64, 5, io, cache, "position", pad=16, gap=2)
    c.run(lse=False)
    c.check(lse=False)
    assert (c.lse == 3.0).all()
    c = Call([40, 3, 129], 6, 2, 64, 5, io, cache, "head", pad=16, gap=2)
    c.run(out=c.tq)  # in place of the queries
    c.check(out=c.tq)


@pytest.mark.parametrize("io,cache", TYPES)
@pytest.mark.parametrize("hd", [128, 32])
def test_sharp_and_large_scores(io, cache, hd):
    """One position takes nearly all the weight; scores of hundreds; a negative scale."""
    for scale, q in ((1.0, 6.0), (-0.5, 3.0), (0.0, 1.0), (1e-4, 1.0)):
        c = Call([200, 1, 64], 4, 2, hd, 16, io, cache, q_scale=q, scale=scale)
        c.run()
        c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("f16", "f16", 64), ("bf16", "bf16", 128), ("f32", "f32", 64), ("f32", "f16", 80), ("f32", "bf16", 64)])
def test_small_and_large_queries_keep_their_digits(io, cache, hd):
    """Queries far from 1 (2^-12 and 2^11 times as large) with scales that undo it."""
    for f in (2.0 ** -12, 2.0 ** 11):
        c = Call([300, 77], 4, 2, hd, 16, io, cache, q_scale=2 * f, scale=1 / (f * math.sqrt(hd)))
        c.run()
        c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("bf16", "bf16", 64), ("f32", "f32", 32), ("f32", "bf16", 80)])
def test_non_finite_values_stay_where_they_reach(io, cache, hd):
    inf, nan = math.inf, math.nan

    def one(change, lens=(70, 5)):
        c = Call(list(lens), 2, 1, hd, 16, io, cache)
        change(c)
        c.run()
        torch.cuda.synchronize()
        return c.out[:, :2 * hd].float().cpu().view(-1, 2, hd), c.lse.cpu()

    def put(c, t, b, j, d, x):
        page = int(c.c.table[b, j // 16])
        t[page, 0, j % 16, d] = x

    o, l = one(lambda c: put(c, c.c.tk, 0, 69, 3, nan))
    assert o[0].isnan().all() and l[0].isnan().all() and o[1].isfinite().all() and l[1].isfinite().all()
    o, l = one(lambda c: put(c, c.c.tv, 0, 20, 3, nan))
    assert o[0, :, 3].isnan().all() and o[0, :, :3].isfinite().all() and l[0].isfinite().all() and o[1].isfinite().all()
    o, l = one(lambda c: put(c, c.c.tv, 0, 20, 3, inf))
    assert not o[0, :, 3].isfinite().any() and o[0, :, 4:].isfinite().all() and l[0].isfinite().all() and o[1].isfinite().all()

    def infinite(sign):
        def change(c):
            c.tq[:2, :2 * hd] = c.tq[:2, :2 * hd].abs() + 0.1
            put(c, c.c.tk, 0, 20, 3, sign * inf)
        return change
    for sign in (1, -1):
        o, l = one(infinite(sign))
        assert o[1].isfinite().all() and l[1].isfinite().all()
    assert one(infinite(1))[0][0].isnan().all()  # inf / inf

    def all_minus(c):  # every score -inf: 0 / 0
        c.tq[:2, :2 * hd] = c.tq[:2, :2 * hd].abs() + 0.1
        for j in range(5):
            put(c, c.c.tk, 1, j, 3, -inf)
    o, l = one(all_minus)
    assert o[1].isnan().all() and o[0].isfinite().all()
    q_nan = lambda c: c.tq.__setitem__((0, 1), nan)  # noqa: E731
    o, l = one(q_nan)
    assert o[0, 0].isnan().all() and o[0, 1].isfinite().all() and o[1].isfinite().all()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("bf16", "bf16", 64), ("f32", "f32", 32), ("f16", "f16", 80)])
def test_bad_pages_and_lengths_are_reported_and_never_read(io, cache, hd):
    from qwen2_decoder_forward_decode_gb300 import binding
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        c = Call([100, 40], 4, 2, hd, 16, io, cache)
        c.c.ttable[0, 2] = bad  # positions 32 .. 47 of sequence 0 are left out
        keep = [j for j in range(100) if not 32 <= j < 48]
        c.run()
        c.check(err=binding.DEV_PAGE, kv=lambda b, h: (c.c.k[b][keep, h], c.c.v[b][keep, h]) if b == 0 else (c.c.k[b][:, h], c.c.v[b][:, h]))
    c = Call([112, 40], 4, 2, hd, 16, io, cache)  # every entry of the row in use
    c.c.tlens[0] = 10 ** 9
    c.c.tlens[1] = -3
    c.c.lens = [112, 0]
    c.run()
    c.check(err=binding.DEV_PAGE, kv=lambda b, h: (c.c.k[b][:c.c.lens[b], h], c.c.v[b][:c.c.lens[b], h]))
    c = Call([5], 4, 2, hd, 16, io, cache)
    c.c.ttable[0, 0] = c.c.n_pages  # nothing is left
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == binding.DEV_PAGE


@pytest.mark.parametrize("io,cache", [("f32", "f16"), ("f32", "f32")])
def test_offsets_beyond_32_bits(io, cache):
    """Pages more than 2^32 elements apart."""
    from qwen2_decoder_forward_decode_gb300 import binding
    c = Call([40], 4, 2, 64, 16, io, cache)
    stride = 2 ** 30 + 2 ** 12
    esize = c.c.tk.element_size()
    big = torch.zeros(5 * stride + 2 * 16 * 64 * 2, dtype=c.c.tk.dtype, device="cuda")
    tv_at = 16 * 64 * 2
    src = [int(p) for p in c.c.table[0, :3]]
    for to, p in zip((5, 0, 4), src):
        big[to * stride:to * stride + tv_at] = c.c.tk[p].reshape(-1)
        big[to * stride + tv_at:to * stride + 2 * tv_at] = c.c.tv[p].reshape(-1)
    c.c.kv = binding.PagedKV(big.data_ptr(), big.data_ptr() + tv_at * esize, ref.CODE[cache], 6, 16, 2, 64, stride, 1024, 64)
    c.c.ttable[0, :3] = torch.tensor([5, 0, 4], dtype=torch.int32)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("bf16", "bf16", 64), ("f32", "f32", 32)])
def test_calls_repeat_bit_by_bit_and_leave_the_workspace_ready(io, cache, hd):
    a = Call([3000, 5, 0, 700], 12, 2, hd, 16, io, cache)
    b = Call([10, 2500], 12, 2, hd, 16, io, cache, seed=9)
    b.ws = a.ws
    first = None
    for _ in range(3):
        a.out.fill_(3.0)
        a.run()
        b.run()
        a.check()
        b.check()
        got = a.out.clone()
        assert first is None or torch.equal(got[:4], first[:4])
        first = got


def test_two_streams_with_their_own_workspaces():
    calls = [Call([900 + i, 40, 3000], 12, 2, 128, 16, "f32", "f16", seed=i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                c.run()
    for c in calls:
        c.check()


def test_a_captured_call_follows_the_device_lengths_and_tables():
    c = Call([300, 1000, 17], 12, 2, 128, 16, "f32", "f16", blocks=70)
    c.run()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for lens in ([300, 1000, 17], [1, 0, 16], [299, 640, 17], [0, 0, 0], [16, 1000, 1]):
        c.c.tlens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.c.lens = lens
        c.out.fill_(3.0)
        g.replay()
        c.check(kv=lambda b, h: (c.c.k[b][:lens[b], h], c.c.v[b][:lens[b], h]))


@pytest.mark.parametrize("io,cache", TYPES)
@pytest.mark.parametrize("nq,hd", [(16, 32), (9, 8), (40, 16)])
def test_large_groups_of_short_heads_stay_in_their_workspace(io, cache, nq, hd):
    """Split units of groups above 8 heads and at most 32 dimensions, whose parts are padded to 64."""
    c = Call([9000, 3, 0, 4000], nq, 1, hd, 16, io, cache)
    size = c.ws.numel()
    c.ws = torch.cat([c.ws, torch.full((1 << 20,), 77, dtype=torch.uint8, device="cuda")])
    for _ in range(2):
        c.run()
        c.check()
    assert (c.ws[size:] == 77).all() and (c.ws[:16384] == 0).all()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("f32", "f16", 32), ("f32", "bf16", 64), ("f32", "bf16", 128), ("f32", "f32", 64), ("f32", "f16", 256), ("f32", "f32", 256)])
@pytest.mark.parametrize("nq", [4, 20])
@pytest.mark.parametrize("e", [-124, -101, -99, 99, 101, 119])
def test_queries_of_any_exponent(io, cache, hd, nq, e):
    """Queries of 2^e, with scales that undo it: finite scores of finite numbers, near the ends of fp32's range too."""
    c = Call([300, 77], nq, 2, hd, 16, io, cache, q_scale=2.0 ** (e + 1), scale=float(np.float32(2.0 ** -e / math.sqrt(hd))))
    c.run()
    c.check()


@pytest.mark.parametrize("hd,nq", [(64, 4), (128, 4), (64, 20), (256, 4)])
@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("e_k,e_q", [(112, -112), (115, 0), (-110, 0), (-100, 110)])
def test_keys_of_any_exponent(cache, hd, nq, e_k, e_q):
    """Keys of 2^e_k under queries of 2^e_q, with scales that undo both."""
    c = Call([300, 77], nq, 2, hd, 16, "f32", cache, q_scale=2.0 ** (e_q + 1), scale=float(np.float32(2.0 ** -(e_k + e_q) / math.sqrt(hd))))
    c.c.tk.mul_(2.0 ** e_k)  # (a power of two: exact)
    c.c.k = [k * 2.0 ** e_k for k in c.c.k]
    c.run()
    c.check()


def test_zero_and_subnormal_queries():
    for cache in ("f16", "bf16", "f32"):
        c = Call([300, 77], 4, 2, 64, 16, "f32", cache, q_scale=2.0 ** -130, scale=2.0 ** 126)
        c.tq[1] = 0.0
        c.q[1] = 0.0
        c.run()
        c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("bf16", "bf16", 64), ("f16", "f16", 32), ("f32", "bf16", 128), ("f32", "f32", 32), ("f32", "f32", 256), ("bf16", "bf16", 256)])
@pytest.mark.parametrize("nq", [4, 20])
def test_a_sequence_with_no_page_left_is_empty(io, cache, hd, nq):
    """Tables without a page of the cache, of one tile and of many CTAs, give what length 0 gives; a long sequence with
    only its last page keeps that one."""
    from qwen2_decoder_forward_decode_gb300 import binding
    lens = [5000, 40, 5, 3000, 4000, 0]
    c = Call(lens, nq, 2, hd, 16, io, cache)
    c.c.ttable[0] = -7
    c.c.ttable[2] = c.c.n_pages
    c.c.ttable[4, :249] = 10 ** 6
    c.run()
    kept = {0: slice(0), 2: slice(0), 4: slice(3984, 4000)}
    c.check(err=binding.DEV_PAGE, kv=lambda b, h: (c.c.k[b][kept.get(b, slice(None)), h], c.c.v[b][kept.get(b, slice(None)), h]))
    assert (c.out[[0, 2, 5], :nq * hd] == 0).all() and (c.lse[[0, 2, 5]] == -math.inf).all()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("bf16", "bf16", 64), ("f32", "f32", 32)])
def test_scores_of_minus_infinity_are_no_empty_sequence(io, cache, hd):
    """Every score -inf where positions are there, next to pages that are left out: still 0 / 0."""
    from qwen2_decoder_forward_decode_gb300 import binding
    c = Call([3000, 40], 2, 1, hd, 16, io, cache)
    c.tq[:2, :2 * hd] = c.tq[:2, :2 * hd].abs() + 0.1
    c.c.ttable[0, 1:] = -1
    c.c.tk[int(c.c.table[0, 0]), 0, :, 3] = -math.inf
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == binding.DEV_PAGE
    assert c.out[0, :2 * hd].isnan().all() and c.out[1, :2 * hd].isfinite().all()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("bf16", "bf16", 64), ("f32", "f32", 32)])
def test_the_largest_scale_leaves_scores_of_zero(io, cache, hd):
    """Queries of 0 have scores of 0 under any scale: the mean of the values."""
    c = Call([300, 77], 4, 2, hd, 16, io, cache, scale=2.0 ** 127)
    c.tq[:2, :4 * hd] = 0.0
    c.q[:] = 0.0
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("f32", "f32", 32)])
def test_scores_of_minus_infinity_weigh_nothing_next_to_others(io, cache, hd):
    """A long sequence whose scores are -inf but for one page: tiles, warps and blocks without a finite score are joined to one
    with some; another without any score of its own but -inf, next to pages that are left out, in many blocks."""
    from qwen2_decoder_forward_decode_gb300 import binding
    c = Call([6000, 6000, 40], 4, 2, hd, 16, io, cache)
    c.tq[:3, :4 * hd] = c.tq[:3, :4 * hd].abs() + 0.1
    c.q = c.tq[:3, :4 * hd].double().cpu().numpy().reshape(3, 4, hd)
    kept = slice(3 * 16, 4 * 16)
    if cache == "f32":  # (products with the lower pieces of 16-bit caches give NaN for infinite keys)
        for j, page in enumerate(c.c.table[0]):
            if j != 3:
                c.c.tk[int(page), :, :, 3] = -math.inf
    else:
        c.c.ttable[0, :3], c.c.ttable[0, 4:375] = -1, -1
    c.c.ttable[1, :370] = -1
    for page in c.c.table[1, 370:375]:
        c.c.tk[int(page), :, :, 3] = -math.inf
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == binding.DEV_PAGE and c.out[1, :4 * hd].isnan().all()
    c.c.k[1], c.c.v[1] = c.c.k[1][:0], c.c.v[1][:0]
    c.out[1, :4 * hd], c.lse[1] = 0.0, -math.inf  # (checked above; the others by the formula)
    c.check(err=binding.DEV_PAGE, kv=lambda b, h: (c.c.k[b][kept if b == 0 else slice(None), h], c.c.v[b][kept if b == 0 else slice(None), h]))


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("f32", "f32", 32)])
def test_a_long_table_of_no_pages_takes_no_longer_than_one_of_pages(io, cache, hd):
    """2^22 positions in pages of one, all outside the cache, and as many in the one page that it has."""
    from qwen2_decoder_forward_decode_gb300 import binding
    c = Call([1], 2, 1, hd, 1, io, cache, blocks=1 << 22)
    c.c.tlens[0] = 1 << 22
    took = []
    for page in (int(c.c.table[0, 0]), -1):
        c.c.ttable.fill_(page)
        for _ in range(2):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            c.run()
            b.record()
            torch.cuda.synchronize()
        took.append(a.elapsed_time(b))
    assert int(c.err) == binding.DEV_PAGE and (c.out[0] == 0).all() and (c.lse[0] == -math.inf).all()
    assert took[1] < 2 * took[0] + 1, took
