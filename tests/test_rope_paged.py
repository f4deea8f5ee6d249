"""Rotary positions with the append to a paged cache, against the formula in 64 bits."""
import math

import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Step:
    """n tokens with shuffled slots in a cache of NaN; q, k and v in one fused row or apart."""

    def __init__(self, n, nq, nkv, hd, rot, adjacent, io, cache, page=16, layout="head", first=0, scaling="none", fused=True, in_place=False, gap=0, seed=0, scale=1.0):
        from qwen2_decoder_forward_decode_gb300 import binding
        rng = np.random.default_rng(seed + n * 7 + hd)
        self.dims = n, nq, nkv, hd, rot, adjacent, io, cache, page
        self.c = ref.PagedCache(rng, [], nkv, hd, page, cache, layout, spare=ref.pages_of(n, page) + 2, gap=gap)
        x = torch.from_numpy(scale * rng.standard_normal((n, nq + 2 * nkv, hd))).to(ref.torch_dtype(io))
        self.x = x.double().numpy()
        self.fused, self.in_place = fused, in_place
        wide = (nq + 2 * nkv) * hd + (16 if fused else 0)
        buf = torch.full((n, wide), 7.0, dtype=ref.torch_dtype(io))
        buf[:, :(nq + 2 * nkv) * hd] = x.reshape(n, -1)
        self.buf = buf.cuda()
        self.parts = [x[:, :nq].contiguous().cuda(), x[:, nq:nq + nkv].contiguous().cuda(), x[:, nq + nkv:].contiguous().cuda()]
        self.positions = np.arange(first, first + n) if n > 1 else np.array([first])
        self.slots = rng.permutation(self.c.n_pages * page)[:n].astype(np.int64)
        self.turns, self.mscale = binding.rope_turns(rot, 1e6, scaling, 4.0, 4096)
        self.freqs = self.turns.astype(np.float64) / 2.0 ** 64 * 2 * math.pi
        self.tturns = torch.from_numpy(self.turns.view(np.int64)).cuda()
        self.q_out = torch.full((n + 1, nq * hd), 5.0, dtype=ref.torch_dtype(io), device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        from qwen2_decoder_forward_decode_gb300 import binding
        n, nq, nkv, hd, rot, adjacent, io, cache, page = self.dims
        self.tpos, self.tslots = torch.from_numpy(self.positions.astype(np.int32)).cuda(), torch.from_numpy(self.slots).cuda()
        torch.cuda.synchronize()
        e = self.buf.element_size()
        if self.fused:
            q, row = self.buf.data_ptr(), self.buf.shape[1]
            src = [(q, row), (q + nq * hd * e, row), (q + (nq + nkv) * hd * e, row)]
        else:
            src = [(t.data_ptr(), t[0].numel()) for t in self.parts]
        out = src[0] if self.in_place else (self.q_out.data_ptr(), nq * hd)
        binding.rope_append(self.c.kv, n, nq, ref.CODE[io], self.tpos.data_ptr(), self.tslots.data_ptr(), self.tturns.data_ptr(), rot, adjacent, self.mscale, *src[0], *src[1], *src[2], *out,
                            self.err.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()

    def check(self, err=0):
        n, nq, nkv, hd, rot, adjacent, io, cache, page = self.dims
        assert int(self.err) == err
        y = ref.rope(self.x[:, :nq + nkv], self.positions, self.freqs, adjacent, self.mscale, rot)
        tol = ref.rope_bound(self.x[:, :nq + nkv], adjacent, self.mscale, rot)

        def near(got, want, bound, t):
            assert np.all(np.abs(got - want) <= bound + (ref.EPS_HALF[t] if t != "f32" else 0) * (np.abs(want) + bound) + ref.TINY[t])

        if self.in_place:
            got = self.buf[:, :nq * hd] if self.fused else self.parts[0].reshape(n, -1)
        else:
            got = self.q_out[:n]
            assert (self.q_out[n:] == 5.0).all()
        near(got.double().cpu().numpy().reshape(n, nq, hd), y[:, :nq], tol[:, :nq], io)
        tk, tv = self.c.tk.cpu(), self.c.tv.cpu()
        seen = torch.zeros(self.c.n_pages * page, dtype=torch.bool)
        for t, slot in enumerate(self.slots.tolist()):
            if not 0 <= slot < self.c.n_pages * page:
                continue
            seen[slot] = True
            near(self.c.row(tk, slot).double().numpy(), y[t, nq:], tol[t, nq:], cache)
            want = torch.from_numpy(self.x[t, nq + nkv:]).to(ref.torch_dtype(cache))
            assert torch.equal(self.c.row(tv, slot), want)
            self.c.row(tk, slot)[:] = float("nan")
            self.c.row(tv, slot)[:] = float("nan")
        assert torch.isnan(tk).all() and torch.isnan(tv).all(), "written outside the slots"


@pytest.mark.parametrize("io,cache", [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("adjacent", [0, 1])
@pytest.mark.parametrize("n,nq,nkv,hd,rot,page,layout,first,scaling", [
    (1, 12, 2, 128, 128, 16, "head", 177, "none"),
    (16, 12, 2, 128, 64, 16, "position", 3000, "linear"),
    (33, 14, 2, 64, 64, 1, "head", 0, "yarn"),
    (300, 3, 1, 32, 24, 7, "position", 130000, "bands"),
    (77, 4, 4, 96, 72, 64, "head", 5000, "ntk"),
    (9, 5, 1, 8, 2, 3, "position", 1, "none"),
    (20, 2, 2, 256, 256, 16, "head", 9, "none"),
    (70, 9, 3, 80, 40, 16, "head", 70000, "none"),
])
def test_rope_append_matches_the_formula(io, cache, adjacent, n, nq, nkv, hd, rot, page, layout, first, scaling):
    s = Step(n, nq, nkv, hd, rot, adjacent, io, cache, page, layout, first, scaling)
    s.run()
    s.check()


@pytest.mark.parametrize("first", [2 ** 31 - 20, -(2 ** 31), -9, 10 ** 9])
def test_far_and_negative_positions(first):
    """The angle's fraction of a turn is exact in 64 bits; the reference takes it from whole numbers too."""
    s = Step(20, 4, 2, 64, 64, 0, "f32", "f32", first=first)
    pos = s.positions.astype(object)
    frac = np.array([[float(((int(p) * int(w) + 2 ** 63) % 2 ** 64) - 2 ** 63) / 2.0 ** 64 for w in s.turns] for p in pos])
    s.run()
    n, nq, nkv, hd, rot, adjacent, *_ = s.dims
    x = s.x[:, :nq]
    c, sn = np.cos(2 * math.pi * frac)[:, None], np.sin(2 * math.pi * frac)[:, None]
    want = np.concatenate([x[..., :32] * c - x[..., 32:] * sn, x[..., :32] * sn + x[..., 32:] * c], -1)
    got = s.q_out[:n].double().cpu().numpy().reshape(n, nq, hd)
    assert np.all(np.abs(got - want) <= ref.rope_bound(x, 0, 1.0, 64))


@pytest.mark.parametrize("io,cache", [("f32", "f16"), ("bf16", "bf16")])
def test_in_place_queries_and_separate_rows(io, cache):
    for fused in (True, False):
        s = Step(40, 6, 2, 64, 64, 0, io, cache, in_place=True, fused=fused, gap=1)
        s.run()
        s.check()


def test_padded_and_bad_slots_write_nothing():
    from qwen2_decoder_forward_decode_gb300 import binding
    s = Step(24, 4, 2, 64, 64, 0, "f32", "f16")
    s.slots[::5] = -1
    s.run()
    s.check()
    for bad in (-2, s.c.n_pages * 16, 2 ** 62):
        s = Step(24, 4, 2, 64, 64, 0, "f32", "f16")
        s.slots[7] = bad
        s.run()
        s.check(err=binding.DEV_PAGE)


def test_values_beyond_fp16_are_reported():
    from qwen2_decoder_forward_decode_gb300 import binding
    for part in range(3):  # (fp32 queries cannot overflow)
        s = Step(3, 4, 2, 64, 64, 0, "f32", "f16")
        s.buf[1, [0, 4, 6][part] * 64 + 5] = 1e6
        s.run()
        assert int(s.err) == (0 if part == 0 else binding.DEV_RANGE)
    s = Step(3, 4, 2, 64, 64, 0, "f32", "f16")
    s.buf[1, 6 * 64] = float("nan")
    s.run()
    assert int(s.err) == binding.DEV_RANGE
    s = Step(3, 4, 2, 64, 64, 0, "f16", "f16", first=1)
    s.buf[1, 0] = s.buf[1, 32] = 60000.0  # rotated by 2 radians: |a'| > 65504
    s.run()
    assert int(s.err) == binding.DEV_RANGE


def test_on_another_stream_and_captured():
    s = Step(50, 12, 2, 128, 128, 0, "f32", "f16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    s.check()


@pytest.mark.parametrize("io,cache", [("f32", "f32"), ("f32", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("adjacent", [0, 1])
@pytest.mark.parametrize("n,nq,nkv,hd,rot,in_place", [(2000, 12, 2, 64, 64, True), (700, 64, 8, 128, 2, False), (3, 300, 60, 256, 64, False), (40, 128, 128, 72, 72, True), (1217, 2, 1, 16, 6, False)])
def test_more_tokens_than_blocks_and_more_heads_than_threads(io, cache, adjacent, n, nq, nkv, hd, rot, in_place):
    """Several tokens a block, in a ring; more elements of a token than the ring has places."""
    s = Step(n, nq, nkv, hd, rot, adjacent, io, cache, in_place=in_place)
    s.run()
    s.check()
