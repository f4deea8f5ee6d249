"""Attention of groups that share a beginning over a paged cache, against the softmax formula in 64 bits."""
import math

import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
TYPES = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")]
NO_PAGE = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Call:
    """groups: (shared positions, [positions of each sequence in all]). Only the first table of a group holds the shared pages,
    the others hold none there, unless the sequence is too short to share."""

    def __init__(self, groups, nq, nkv, hd, page, io, cache, layout="head", seed=0, q_scale=2.0, pad=0, scale=None, poison=True, **kw):
        from qwen2_decoder_forward_decode_gb300 import binding
        rng = np.random.default_rng(seed + len(groups) + hd)
        self.nq, self.nkv, self.hd, self.io, self.cache = nq, nkv, hd, io, cache
        size = [len(g[1]) for g in groups]
        self.cu = np.concatenate([[0], np.cumsum(size)]).astype(np.int32)
        self.lens = [n for g in groups for n in g[1]]
        self.shared = np.repeat([g[0] for g in groups], size).astype(np.int32)
        first = np.repeat(self.cu[:-1], size)
        n = len(self.lens)
        # the first sequence's table holds the shared part whatever its own length is
        held = [max(m, int(self.shared[b])) if b == first[b] else m for b, m in enumerate(self.lens)]
        c = self.c = ref.PagedCache(rng, held, nkv, hd, page, cache, layout, **kw)
        for b in range(n):
            p = int(self.shared[b])
            if b == first[b] or self.lens[b] < p or not p:
                continue
            for arr, t in ((c.k, c.tk), (c.v, c.tv)):
                arr[b][:p] = arr[first[b]][:p]
                for j in range(p // page, ref.pages_of(min(p, self.lens[b]), page)):  # the page on which it ends, as a fork copies it
                    m = p - j * page
                    src, dst = t[int(c.table[first[b], j])], t[int(c.table[b, j])]
                    if layout == "head":
                        dst[:, :m] = src[:, :m]
                    else:
                        dst[:m] = src[:m]
            if poison:
                c.table[b, :p // page] = NO_PAGE
        c.ttable = torch.from_numpy(c.table).cuda()
        self.tlens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.tcu, self.tshared = torch.from_numpy(self.cu).cuda(), torch.from_numpy(self.shared).cuda()
        q = torch.from_numpy(q_scale * rng.standard_normal((n, nq, hd))).to(ref.torch_dtype(io))
        self.tq = torch.full((n + 1, nq * hd + pad), float("nan"), dtype=q.dtype)  # (one more row than sequences)
        self.tq[:n, :nq * hd] = q.reshape(n, -1)
        self.tq = self.tq.cuda()
        self.out = torch.full_like(self.tq, 3.0)
        self.lse = torch.full((n + 1, nq), 3.0, device="cuda")
        self.scale = 1 / math.sqrt(hd) if scale is None else scale
        self.ws = torch.zeros(binding.shared_attention_workspace(n, nq, nkv, hd), dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, out=None, lse=True):
        from qwen2_decoder_forward_decode_gb300 import binding
        out = self.out if out is None else out
        binding.shared_attention(self.c.kv, len(self.lens), self.nq, self.c.ttable.data_ptr(), self.c.blocks, self.tlens.data_ptr(), len(self.cu) - 1, self.tcu.data_ptr(), self.tshared.data_ptr(),
                                 ref.CODE[self.io], self.tq.data_ptr(), self.tq.shape[1], self.scale, out.data_ptr(), out.shape[1], self.lse.data_ptr() if lse else None, self.ws.data_ptr(),
                                 self.ws.numel(), self.err.data_ptr(), torch.cuda.current_stream().cuda_stream)

    def got(self, out=None):
        torch.cuda.synchronize()
        n = len(self.lens)
        out = (self.out if out is None else out).double().cpu().numpy()
        assert (out[n:] == 3.0).all() or np.isnan(out[n:]).all()
        assert (self.lse[n:] == 3.0).all()
        return out[:n, :self.nq * self.hd].reshape(n, self.nq, self.hd), self.lse.double().cpu().numpy()[:n]

    def check(self, out=None, err=0, lse=True, only=None, q=None):
        got, tl = self.got(out)
        assert int(self.err) == err
        g = self.nq // self.nkv
        q = self.tq.double().cpu().numpy()[:len(self.lens), :self.nq * self.hd].reshape(got.shape) if q is None else q
        for b in range(len(self.lens)) if only is None else only:
            for h in range(self.nkv):
                k, v = self.c.k[b][:self.lens[b], h], self.c.v[b][:self.lens[b], h]
                heads = slice(h * g, (h + 1) * g)
                o, l, bound = ref.attention(q[b, heads], k, v, self.scale)
                if self.io != "f32" and len(k):  # a 16-bit caller's probabilities are rounded once to the cache's type, fp16 ones
                    z = self.scale * (q[b, heads] @ k.T)  # times 2^10: normal down to 2^-24 of the largest
                    p = np.exp(z - z.max(-1, keepdims=True))
                    bound = bound + ref.EPS_HALF[self.cache] * (p / p.sum(-1, keepdims=True)) @ np.abs(v)
                    if self.cache == "f16":
                        bound = bound + 2.0 ** -35 / p.sum(-1, keepdims=True) * np.abs(v).sum(0)
                tol = bound + (ref.EPS_HALF[self.io] if self.io != "f32" else 0) * (np.abs(o) + bound) + ref.TINY[self.io]
                np.testing.assert_array_less(np.abs(got[b, heads] - o), tol + 1e-30, err_msg=f"sequence {b} KV head {h} length {self.lens[b]}")
                if lse:
                    ds = (8 * math.sqrt(self.hd) + 4) * ref.U * abs(self.scale) * (np.abs(q[b, heads]) @ np.abs(k).T).max(initial=0)
                    with np.errstate(invalid="ignore"):
                        off = np.where(l == tl[b, heads], 0.0, np.abs(tl[b, heads] - l))
                    assert np.all(off <= ds + (8 * math.sqrt(len(k)) + 8) * ref.U + ref.U * np.where(np.isfinite(l), np.abs(l), 0)), (b, h)


SHAPES = [(12, 2, 128), (14, 2, 64), (4, 4, 16), (28, 4, 128), (3, 1, 32), (16, 1, 96), (9, 3, 80), (40, 2, 128), (2, 1, 256), (1, 1, 8)]
GROUPS = [(130, [131, 150, 130, 200]), (0, [7, 0, 3]), (1, [1, 2]), (64, [0, 64, 70]), (100, [100, 40, 120, 0, 101]), (300, [400] * 11), (5, [])]


@pytest.mark.parametrize("io,cache", TYPES)
@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("page,layout", [(16, "head"), (7, "position")])
def test_ragged_groups(io, cache, nq, nkv, hd, page, layout):
    c = Call(GROUPS, nq, nkv, hd, page, io, cache, layout)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache", TYPES)
@pytest.mark.parametrize("groups,page", [
    ([(4000, [4001, 4010, 4000])], 16), ([(1, [1])], 1), ([(2500, [2500 + 3 * i for i in range(40)])], 64), ([(127, [128] * 3), (128, [128] * 3), (129, [130] * 3)], 256), ([(1500, [1600] * 30), (900, [901])], 1),
])
def test_long_and_wide_groups(io, cache, groups, page):
    c = Call(groups, 12, 2, 128, page, io, cache)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 64), ("bf16", "bf16", 128), ("f32", "f32", 32), ("f32", "bf16", 128)])
def test_many_groups(io, cache, hd):
    """More groups than a CTA has threads, some of them empty."""
    rng = np.random.default_rng(4)
    groups = [(int(rng.integers(0, 200)), [0] * int(rng.integers(0, 4))) for _ in range(600)]
    groups = [(p, [p + int(rng.integers(0, 9)) for _ in g]) for p, g in groups]
    c = Call(groups, 4, 2, hd, 16, io, cache)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache", TYPES)
def test_a_very_long_beginning(io, cache):
    c = Call([(70000, [70001, 70000, 70100])], 4, 1, 64, 16, io, cache)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache", TYPES)
def test_strides_gaps_in_place_and_no_lse(io, cache):
    c = Call([(40, [50, 41]), (129, [129])], 6, 2, 64, 5, io, cache, "position", pad=16, gap=2)
    q = c.tq.double().cpu().numpy()[:3, :6 * 64].reshape(3, 6, 64)
    c.run(lse=False)
    c.check(lse=False)
    assert (c.lse == 3.0).all()
    c.run(out=c.tq)
    c.check(out=c.tq, q=q)


@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0, 1e-30])
@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 64), ("bf16", "bf16", 128), ("f32", "f32", 32), ("f32", "bf16", 128)])
def test_scales_of_any_sign(io, cache, hd, scale):
    c = Call([(200, [201, 230, 200]), (31, [40])], 8, 2, hd, 16, io, cache, scale=scale)
    c.run()
    c.check()


@pytest.mark.parametrize("e", [-120, -30, 0, 30, 90])
@pytest.mark.parametrize("cache,hd", [("f16", 64), ("bf16", 128), ("f32", 32)])
def test_queries_of_any_exponent(cache, hd, e):
    c = Call([(300, [301, 320])], 6, 2, hd, 16, "f32", cache, q_scale=2.0 ** e, scale=2.0 ** -e / math.sqrt(hd))
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 64), ("bf16", "bf16", 128), ("f32", "f32", 32), ("f16", "f16", 128)])
def test_groups_give_what_sequences_alone_give(io, cache, hd):
    """The operator over tables that hold all positions, next to qw_op_paged_attention on the same."""
    from qwen2_decoder_forward_decode_gb300 import binding
    c = Call([(500, [501 + 7 * i for i in range(9)]), (64, [65, 64])], 12, 2, hd, 16, io, cache, poison=False)
    first = np.repeat(c.cu[:-1], np.diff(c.cu))
    for b in range(len(c.lens)):
        c.c.table[b, :int(c.shared[b]) // 16] = c.c.table[first[b], :int(c.shared[b]) // 16]
    c.c.ttable.copy_(torch.from_numpy(c.c.table))
    c.run()
    c.check()
    out, lse = torch.full_like(c.out, 3.0), torch.zeros_like(c.lse)
    n = len(c.lens)
    binding.paged_attention(c.c.kv, n, c.nq, c.c.ttable.data_ptr(), c.c.blocks, c.tlens.data_ptr(), ref.CODE[io], c.tq.data_ptr(), c.tq.shape[1], c.scale, out.data_ptr(), out.shape[1], lse.data_ptr(),
                            c.ws.data_ptr(), c.ws.numel(), c.err.data_ptr(), torch.cuda.current_stream().cuda_stream)  # (a workspace of this operator serves that one)
    c.check(out=out, lse=False)
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("bf16", "bf16", 64), ("f32", "f32", 32)])
def test_non_finite_values_stay_where_they_reach(io, cache, hd):
    nan, inf = float("nan"), float("inf")
    c = Call([(200, [210, 150, 200, 0]), (100, [130, 120])], 4, 2, hd, 16, io, cache)
    layout_row = lambda t, b, pos: c.c.row(t, int(c.c.table[b, pos // 16]) * 16 + pos % 16)  # noqa: E731
    layout_row(c.c.tk, 0, 100)[0, 3] = nan   # shared by sequences 0 and 2, KV head 0; sequence 1 reads its own pages
    layout_row(c.c.tv, 4, 50)[1, 2] = inf    # shared by 4 and 5, KV head 1, dimension 2
    layout_row(c.c.tk, 5, 115)[0, 1] = nan   # sequence 5's own
    c.tq[2, 3 * hd] = nan                    # a query of sequence 2, head 3
    c.run()
    got, lse = c.got()
    assert int(c.err) == 0
    assert np.isnan(got[[0, 2], :2]).all() and np.isnan(lse[[0, 2], :2]).all()
    assert np.isfinite(got[0, 2:]).all() and np.isfinite(got[2, 2]).all() and np.isnan(got[2, 3]).all()
    # (an infinite value makes an output infinite or NaN: a probability's lower piece may be 0 or negative)
    assert not np.isfinite(got[4:6, 2:, 2]).any() and np.isfinite(np.delete(got[4:6, 2:], 2, -1)).all()
    assert np.isnan(got[5, :2]).all() and np.isfinite(got[4, :2]).all()
    assert (got[3] == 0).all() and np.isneginf(lse[3]).all()
    q = c.tq.double().cpu().numpy()[:6, :4 * hd].reshape(got.shape)
    c.check(only=[1], q=q)


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 64), ("bf16", "bf16", 128), ("f32", "f32", 32)])
def test_bad_pages_are_left_out(io, cache, hd):
    c = Call([(100, [110, 105]), (40, [40, 50])], 4, 2, hd, 16, io, cache)
    c.c.ttable[0, 2] = -1
    c.c.ttable[2, 0] = c.c.n_pages
    c.c.ttable[2, 1:3] = c.c.n_pages + 5   # nothing is left of the second group's beginning
    c.run()
    for b in (0, 1):
        for arr in (c.c.k, c.c.v):
            arr[b] = np.delete(arr[b], np.s_[32:48], axis=0)
        c.lens[b] -= 16
    for arr in (c.c.k, c.c.v):
        arr[2], arr[3] = arr[2][:0], arr[3][40:]
    c.lens[2:] = [0, 10]
    c.check(err=32)


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 64), ("f32", "f32", 32)])
@pytest.mark.parametrize("cu", [[0, 2, 5], [1, 2, 4], [0, 3, 2], [0, -1, 4], [0, 2, 3], [0, 9, 4]])
def test_bad_groups_give_nothing(io, cache, hd, cu):
    c = Call([(100, [110, 105]), (40, [40, 50])], 4, 2, hd, 16, io, cache)
    c.tcu.copy_(torch.tensor(cu, dtype=torch.int32))
    c.run()
    got, lse = c.got()
    assert int(c.err) & 32 and (got == 0).all() and np.isneginf(lse).all()
    c.err.zero_()
    c.tcu.copy_(torch.from_numpy(c.cu))
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 64), ("f32", "f32", 32), ("bf16", "bf16", 128), ("f32", "f16", 256)])
@pytest.mark.parametrize("cu", [[-(1 << 30), 2, 4], [1 << 30, 2, 4], [0, 1 << 30, 4], [0, -(1 << 30), 4], [0, 2, 1 << 30], [-1, -1, -1]])
def test_bounds_far_out_give_nothing(io, cache, hd, cu):
    c = Call([(100, [110, 105]), (40, [40, 50])], 4, 2, hd, 16, io, cache)
    c.tcu.copy_(torch.tensor(cu, dtype=torch.int32))
    c.run()
    got, lse = c.got()
    assert int(c.err) & 32 and (got == 0).all() and np.isneginf(lse).all()
    c.err.zero_()
    c.tcu.copy_(torch.from_numpy(c.cu))
    c.run()
    c.check()


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 64), ("f32", "f32", 32)])
def test_bad_shared_lengths_are_reported(io, cache, hd):
    c = Call([(100, [110, 105, 103]), (40, [40, 50])], 4, 2, hd, 16, io, cache)
    c.tshared[1] = 96
    c.run()
    c.check(err=32, only=[0, 2, 3, 4])
    for value in (-1, 1 << 30):
        c.err.zero_()
        c.tshared[1] = value
        c.run()
        c.got()
        assert int(c.err) == 32
        c.check(err=32, only=[0, 2, 3, 4])
    c.err.zero_()
    c.tshared[1] = 100
    c.tlens[0] = -3
    c.run()
    c.check(err=32, only=[1, 2, 3, 4])


def test_no_sequences():
    from qwen2_decoder_forward_decode_gb300 import binding
    c = Call([(100, [110])], 4, 2, 64, 16, "f32", "f16")
    binding.shared_attention(c.c.kv, 0, 4, None, 1, None, 0, None, None, 0, None, 256, 1.0, None, 256, None, None, 0, None, None)


def test_offsets_beyond_32_bits():
    """One page of the beginning lies 5 G elements into the cache."""
    from qwen2_decoder_forward_decode_gb300 import binding
    page, nkv, hd = 64, 2, 128
    n_pages = 5 * 2 ** 30 // (page * nkv * hd)
    k, v = (torch.zeros(n_pages, nkv, page, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = [n_pages - 1, 7, n_pages // 2]
    for i in ids:
        k[i].normal_()
        v[i].normal_()
    kv = binding.PagedKV(k.data_ptr(), v.data_ptr(), 1, n_pages, page, nkv, hd, nkv * page * hd, page * hd, hd)
    q = torch.randn(2, 4 * hd, device="cuda").to(torch.bfloat16)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, cu, shared, err = i32(*ids, *ids).view(2, 3), i32(150, 130), i32(0, 2), i32(128, 128), i32(0)
    out, lse = torch.zeros_like(q), torch.zeros(2, 4, device="cuda")
    ws = torch.zeros(binding.shared_attention_workspace(2, 4, nkv, hd), dtype=torch.uint8, device="cuda")
    binding.shared_attention(kv, 2, 4, table.data_ptr(), 3, lens.data_ptr(), 1, cu.data_ptr(), shared.data_ptr(), 1, q.data_ptr(), 4 * hd, 0.1, out.data_ptr(), 4 * hd, lse.data_ptr(), ws.data_ptr(),
                             ws.numel(), err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert int(err) == 0
    for b, n in enumerate((150, 130)):
        for h in range(nkv):
            kk, vv = (torch.cat([t[i, h] for i in ids])[:n].double().cpu().numpy() for t in (k, v))
            qq = q[b].view(4, hd)[2 * h:2 * h + 2].double().cpu().numpy()
            o, _, bound = ref.attention(qq, kk, vv, 0.1)
            z = np.exp(0.1 * (qq @ kk.T))
            bound = bound + 2.0 ** -8 * (z / z.sum(-1, keepdims=True)) @ np.abs(vv)
            np.testing.assert_array_less(np.abs(out[b].view(4, hd)[2 * h:2 * h + 2].double().cpu().numpy() - o), bound + 2.0 ** -8 * (np.abs(o) + bound))


@pytest.mark.parametrize("io,cache,hd", [("f32", "f16", 128), ("bf16", "bf16", 128), ("f32", "f32", 64), ("f32", "bf16", 64)])
def test_calls_repeat_bit_by_bit_captured_and_on_other_streams(io, cache, hd):
    c = Call([(700, [720, 700, 710]), (33, [40] * 20), (0, [300])], 12, 2, hd, 16, io, cache)
    c.run()
    c.check()
    out, lse = c.out.clone(), c.lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for i in range(6):
        c.out.fill_(3.0)
        torch.cuda.synchronize()
        if i % 2:
            g.replay()
        else:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out.view(torch.uint8), out.view(torch.uint8)) and torch.equal(c.lse, lse)
    # the graph follows the lengths, groups and shared positions that the device holds
    c.lens = [705, 700, 20] + [33] * 20 + [299]
    c.tlens.copy_(torch.tensor(c.lens, dtype=torch.int32))
    g.replay()
    c.check(err=32, only=[0, 1, 3, 22, 23])  # (sequence 2 is now too short to share, and its own table has no such pages)


@pytest.mark.parametrize("io,cache,hd,page", [("bf16", "bf16", 128, 64), ("f16", "f16", 64, 16), ("f32", "f16", 128, 64), ("bf16", "bf16", 128, 5)])
def test_many_calls_of_many_units_agree(io, cache, hd, page):
    """Short and long groups of few rows in turn, hundreds of times: a wait that is answered for another tile, or a tile that
    is given back twice, shows as other bits or as a wait that runs out."""
    rng = np.random.default_rng(hd)
    groups = [(int(p), [int(p) + int(rng.integers(0, 40))] * int(rng.integers(1, 3))) for p in rng.integers(1, 1500, 200)]
    c = Call(groups, 28, 4, hd, page, io, cache)
    c.run()
    c.check()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(400):
        c.run()
    torch.cuda.synchronize()
    assert int(c.err) == 0 and torch.equal(c.out.view(torch.uint8), out.view(torch.uint8)) and torch.equal(c.lse, lse)


def test_two_streams_with_their_own_workspaces():
    calls = [Call([(900, [920, 910]), (200, [222] * 9)], 12, 2, 128, 16, "bf16", "bf16", seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    for c in calls:
        c.check()
