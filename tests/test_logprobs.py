"""Token log probabilities, ranks, entropy and top tokens against 64-bit numpy."""
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


class Call:
    def __init__(self, z, dtype, ids, top_k, gap=0, offset=0):
        """z [rows][vocab] numpy; ids [rows][n_ids]; offset: elements before the first row."""
        from qwen2_decoder_forward_decode_gb300 import binding
        t = torch.from_numpy(np.asarray(z, dtype=np.float64)).to(ref.torch_dtype(dtype))
        self.z = t.double().numpy()
        self.rows, self.vocab = t.shape
        self.dtype, self.k, self.stride, self.offset = dtype, top_k, self.vocab + gap, offset
        buf = torch.full((offset + self.rows * self.stride,), float("inf"), dtype=t.dtype)  # gaps that must not count
        buf[offset:].view(self.rows, self.stride)[:, :self.vocab] = t
        self.buf = buf.cuda()
        self.ids = np.asarray(ids, dtype=np.int32).reshape(self.rows, -1)
        self.n_ids = self.ids.shape[1]
        self.tids = torch.from_numpy(self.ids).cuda()
        full = lambda *s, d=torch.float32: torch.full(s, 55, dtype=d, device="cuda")  # noqa: E731
        self.lp, self.ranks, self.ent = full(self.rows + 1, max(self.n_ids, 1)), full(self.rows + 1, max(self.n_ids, 1), d=torch.int32), full(self.rows + 1)
        self.top_ids, self.top_lp = full(self.rows + 1, max(top_k, 1), d=torch.int32), full(self.rows + 1, max(top_k, 1))
        self.ws = torch.zeros(binding.token_logprobs_workspace(self.rows, self.vocab, top_k), dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, ranks=True, entropy=True):
        from qwen2_decoder_forward_decode_gb300 import binding
        p = lambda t, on=True: t.data_ptr() if on else None  # noqa: E731
        binding.token_logprobs(ref.CODE[self.dtype], self.rows, self.vocab, self.buf.data_ptr() + self.offset * self.buf.element_size(), self.stride, p(self.tids, self.n_ids), self.n_ids,
                               p(self.lp, self.n_ids), p(self.ranks, self.n_ids and ranks), p(self.ent, entropy), self.k, p(self.top_ids, self.k), p(self.top_lp, self.k), self.ws.data_ptr(),
                               self.ws.numel(), self.err.data_ptr(), torch.cuda.current_stream().cuda_stream)

    def check(self, err=0, ranks=True, entropy=True):
        torch.cuda.synchronize()
        assert int(self.err) == err
        n = self.rows
        lp, rk, ent, ti, tl = (t.cpu().numpy() for t in (self.lp, self.ranks, self.ent, self.top_ids, self.top_lp))
        for t in (lp, rk, ent, ti, tl):
            assert (t[n:] == 55).all(), "written behind the last row"
        assert ranks or (rk == 55).all()
        assert entropy or (ent == 55).all()
        for r in range(n):
            z = self.z[r]
            ids = self.ids[r]
            in_range = (ids >= 0) & (ids < self.vocab)
            if np.isnan(z).any() or (z == np.inf).any() or (z == -np.inf).all():
                for i, t in enumerate(ids):
                    assert (lp[r, i] == 0 if t == -1 else np.isnan(lp[r, i])) and (not ranks or rk[r, i] == 0)
                assert not entropy or np.isnan(ent[r])
                if self.k:
                    assert (ti[r] == -1).all() and np.isnan(tl[r]).all()
                continue
            m = z.max()
            e = np.exp(z - m)
            S = e.sum()
            ln_s = math.log(S)  # (z - m - ln S, not z - (m + ln S): at 3e38 a step of 64 bits is 4e22)
            p = e / S
            with np.errstate(invalid="ignore"):
                H = math.log(S) - np.sum(np.where(p > 0, p * (z - m), 0.0))
            # S: positive terms summed in at most 400 steps on one path, at 8 standard deviations of half a
            # step, and exponentials good to 2^-22: 8 * 20 * 2^-24 + 2^-22 = 9.8e-6; z - m, ln S and their
            # difference: a step each
            near = lambda got, v: got == np.float32(v - m - ln_s) or abs(got - (v - m - ln_s)) <= tol(v)  # noqa: E731 (beyond fp32: -inf)
            tol = lambda v: 1e-5 + ref.U * (abs(v - m) + abs(math.log(S)))  # noqa: E731
            order = np.lexsort((np.arange(self.vocab), -(z + 0.0)))
            place = np.empty(self.vocab, dtype=np.int64)
            place[order] = np.arange(1, self.vocab + 1)
            for i, t in enumerate(ids):
                if not in_range[i]:
                    assert (lp[r, i] == 0 if t == -1 else np.isnan(lp[r, i])) and (not ranks or rk[r, i] == 0)
                    continue
                assert lp[r, i] == z[t] if z[t] == -np.inf else near(lp[r, i], z[t]), (r, i)
                assert not ranks or rk[r, i] == place[t], (r, i)
            # W / S has the relative errors of both sums, and W / S = ln S - H
            assert not entropy or abs(ent[r] - H) <= 1e-5 * (2 + 2 * abs(H) + abs(math.log(S))), r
            if self.k:
                np.testing.assert_array_equal(ti[r], order[:self.k], err_msg=f"row {r}")
                for i in range(self.k):
                    v = z[order[i]]
                    assert tl[r, i] == v if v == -np.inf else near(tl[r, i], v), (r, i)


def logits(rng, rows, vocab, hot=6):
    z = 2 * rng.standard_normal((rows, vocab))
    for r in range(rows):
        z[r, rng.integers(0, vocab, min(hot, vocab))] += 6
    return z


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab,n_ids,top_k", [
    (1, 151936, 1, 5), (1, 151936, 8, 32), (3, 152064, 2, 20), (1, 1, 1, 1), (2, 2, 1, 2), (5, 32, 3, 32), (7, 33, 0, 32), (40, 1000, 1, 0), (33, 3001, 1, 1), (300, 257, 2, 10),
    (2, 16384, 1, 20), (2, 16385, 1, 20), (6, 32000, 1, 20), (400, 5000, 1, 20), (1, 300001, 2, 32), (170, 32767, 5, 32),
])
def test_rows_match_the_definition(dtype, rows, vocab, n_ids, top_k):
    rng = np.random.default_rng(rows + vocab)
    z = logits(rng, rows, vocab)
    c = Call(z, dtype, rng.integers(0, vocab, (rows, n_ids)), top_k)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gap,offset", [(1, 0), (7, 3), (8, 8), (64, 1)])
def test_strided_and_misaligned_rows(dtype, gap, offset):
    rng = np.random.default_rng(gap)
    c = Call(logits(rng, 9, 4099), dtype, rng.integers(0, 4099, (9, 2)), 12, gap, offset)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [100, 5000, 152064])
@pytest.mark.parametrize("kind", ["equal", "two values", "ascending", "descending", "one finite", "zeros", "masked", "blocks", "late"])
def test_ties_and_orders(dtype, vocab, kind):
    """Rows on which a threshold for the top tokens holds badly: ties, sorted logits, mostly -inf."""
    rng = np.random.default_rng(4)
    j = np.arange(vocab)
    z = {"equal": np.full(vocab, -3.25), "two values": (j % 7 == 5) * 1.0, "ascending": j / vocab * 8, "descending": -(j / vocab) * 8, "one finite": np.where(j == vocab - 2, 1.5, -np.inf),
         "zeros": np.where(j % 2 == 0, -0.0, 0.0), "masked": np.where(j % 50 == 3, rng.standard_normal(vocab), -np.inf), "blocks": (j // 64 % 5) * 0.5,
         "late": np.where(j >= vocab - 40, 5.0 + (j - vocab) / 64, rng.standard_normal(vocab) * 0.1)}[kind]
    c = Call(np.stack([z, z[::-1]]), dtype, [[0, vocab - 2, vocab // 2], [vocab - 1, 1, 1]], 32)
    c.run()
    c.check()


def test_rows_without_a_distribution():
    from qwen2_decoder_forward_decode_gb300 import binding
    rng = np.random.default_rng(0)
    for vocab in (50, 40000):
        z = logits(rng, 6, vocab)
        z[1, 7] = np.nan
        z[2, vocab - 1] = np.inf
        z[3, :] = -np.inf
        z[4, 5] = -np.inf
        c = Call(z, "f32", [[3, -1]] * 6, 4)
        c.run()
        c.check(err=binding.DEV_NONFINITE)


def test_ids_outside_the_vocabulary():
    from qwen2_decoder_forward_decode_gb300 import binding
    rng = np.random.default_rng(0)
    c = Call(logits(rng, 3, 500), "f32", [[3, -1, 3], [-1, -1, 499], [0, 1, 2]], 4)
    c.run()
    c.check()
    for bad in (500, -2, 2 ** 31 - 1, -2 ** 31):
        c = Call(logits(rng, 2, 500), "f32", [[3, bad], [1, 2]], 4)
        c.run()
        c.check(err=binding.DEV_TOKEN)


def test_optional_outputs():
    rng = np.random.default_rng(0)
    for n_ids, k, ranks, entropy in ((0, 0, False, True), (1, 0, False, False), (0, 3, False, False), (2, 3, True, False)):
        c = Call(logits(rng, 4, 20000), "f32", rng.integers(0, 20000, (4, n_ids)), k)
        c.run(ranks, entropy)
        c.check(0, ranks and n_ids > 0, entropy)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [40, 9000, 70001])
def test_rows_masked_with_the_lowest_value(dtype, vocab):
    """Masks of the type's lowest value instead of -inf, alone and next to it, rows that leave nothing, and logits
    so large that their product with log2(e) is not finite."""
    rng = np.random.default_rng(vocab)
    low, high = float(torch.finfo(ref.torch_dtype(dtype)).min), float(torch.finfo(ref.torch_dtype(dtype)).max)
    some = rng.random(vocab) < 0.03
    some[vocab // 2] = True
    z = [np.full(vocab, low), np.where(some, low, -np.inf), np.where(some, rng.standard_normal(vocab), low), np.where(some, low, rng.standard_normal(vocab)),
         np.where(np.arange(vocab) % 3 == 0, -np.inf, np.where(some, 2.0, low)), np.where(some, high, 1.0), np.where(some, high, low), np.where(some, high / 2, high),
         np.where(some, low / 2, low), np.where(some, low * 0.25, -np.inf), np.where(some, high, -np.inf)]
    c = Call(np.stack(z), dtype, [[vocab // 2, 0, vocab - 1, 1]] * len(z), 32)
    c.run()
    c.check()
    z[3][5] = np.nan  # a NaN counts in a row of extreme values too
    z[5][vocab - 3] = np.nan
    z[0][vocab // 3] = np.nan
    from qwen2_decoder_forward_decode_gb300 import binding
    c = Call(np.stack(z), dtype, [[vocab // 2, 0]] * len(z), 3)
    c.run()
    c.check(err=binding.DEV_NONFINITE)


def _short_rows(rng, vocab, kind):
    j = np.arange(vocab)
    return {"random": lambda: rng.standard_normal(vocab) * 2, "equal": lambda: np.full(vocab, -3.25), "two values": lambda: (j % 3 == 1) * 1.0, "ascending": lambda: j / vocab * 8,
            "masked": lambda: np.where(rng.random(vocab) < 0.9, -np.inf, rng.standard_normal(vocab)), "one finite": lambda: np.where(j == vocab // 2, 1.5, -np.inf),
            "tiny": lambda: rng.integers(-3, 4, vocab) * 2.0 ** -23, "nan": lambda: np.where(j == vocab - 1, np.nan, 0.5), "inf": lambda: np.where(j == vocab // 3, np.inf, 0.5),
            "empty": lambda: np.full(vocab, -np.inf), "lowest": lambda: np.where(rng.random(vocab) < 0.5, -65504.0, -np.inf)}[kind]()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab,rows,gap,offset", [(1, 5, 0, 0), (31, 3, 2, 1), (257, 5000, 1, 3), (1024, 700, 0, 0), (1025, 460, 3, 2), (2049, 1000, 0, 5), (4999, 1900, 1, 0), (6143, 3200, 0, 1),
                                                     (6145, 3200, 0, 0), (12287, 3200, 0, 0)])
def test_many_short_rows(dtype, vocab, rows, gap, offset):
    """Rows of a few KB, in numbers where one warp has a row and beyond: the first ones against the definition, the others, their
    repeats, bit by bit against them (8 periods apart: a row's start within 16 bytes decides the order of its sums)."""
    from qwen2_decoder_forward_decode_gb300 import binding
    rng = np.random.default_rng(vocab)
    kinds = ["random", "equal", "two values", "ascending", "masked", "one finite", "tiny", "nan", "inf", "empty", "lowest", "random", "random"]
    n = min(rows, len(kinds))
    z = np.stack([_short_rows(rng, vocab, k) for k in kinds[:n]])
    ids = np.stack([rng.integers(0, vocab, n), rng.integers(0, vocab, n), np.full(n, vocab - 1), np.full(n, -1), np.zeros(n)], axis=1)
    top = min(vocab, 32)
    repeat = np.arange(rows) % n
    c = Call(z[repeat], dtype, ids[repeat], top, gap, offset)
    c.run()
    torch.cuda.synchronize()
    first = min(8 * n, rows)
    # longer rows may be cut, at different places: two results near one truth, each by the bounds of check(), where
    # |ln p| = (m - z) + ln S and ln S, H <= ln vocab
    cut = vocab * c.buf.element_size() > 24576
    for t, bound in ((c.lp, 1e-5), (c.ranks, 0), (c.ent, 1e-5 * (2 + 3 * math.log(vocab))), (c.top_ids, 0), (c.top_lp, 1e-5)):
        got, again = t[:first][torch.arange(first, rows, device="cuda") % first], t[first:rows]
        same = got.view(torch.int32) == again.view(torch.int32)
        if cut and bound:
            same |= (got.double() - again.double()).abs() <= 2 * (bound + ref.U * got.double().abs())
        assert same.all()
        assert (t[rows:] == 55).all()
        t[first:] = 55
    c.rows = first
    odd = any(np.isnan(r).any() or (r == np.inf).any() or (r == -np.inf).all() for r in c.z[:n])
    c.check(err=binding.DEV_NONFINITE if odd else 0)


@pytest.mark.parametrize("dtype,vocab", [("f32", 400003), ("bf16", 800001), ("f32", 4000001)])
@pytest.mark.parametrize("kind", ["random", "ascending", "descending", "equal", "one finite", "few finite"])
def test_a_row_of_many_parts(dtype, vocab, kind):
    """About 50 and 450 parts are joined: lists that all reach the bound, that hardly any does, that are empty."""
    rng = np.random.default_rng(vocab)
    j = np.arange(vocab)
    z = {"random": lambda: rng.standard_normal(vocab), "ascending": lambda: j / vocab * 8, "descending": lambda: j / vocab * -8, "equal": lambda: np.full(vocab, 0.5),
         "one finite": lambda: np.where(j == vocab // 2, 1.5, -np.inf), "few finite": lambda: np.where(j % (vocab // 20) == 7, 0.25, -np.inf)}[kind]()
    c = Call(z[None], dtype, [[0, vocab - 1, vocab // 2, 7, -1]], 32)
    c.run()
    c.check()


def test_large_values():
    rng = np.random.default_rng(0)
    for shift, scale in ((1e4, 1.0), (-3e4, 1.0), (0.0, 300.0)):
        c = Call(shift + scale * rng.standard_normal((3, 30000)), "f32", rng.integers(0, 30000, (3, 1)), 20)
        c.run()
        c.check()


def test_repeats_bit_by_bit_captured_and_on_another_stream():
    rng = np.random.default_rng(1)
    z = logits(rng, 5, 151936)
    c = Call(z, "f32", rng.integers(0, 151936, (5, 2)), 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    c.check()
    first = [t.clone() for t in (c.lp, c.ent, c.top_lp)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for _ in range(3):
        for t in (c.lp, c.ent, c.top_lp, c.ranks, c.top_ids):
            t.fill_(55)
        g.replay()
        c.check()
        assert all(torch.equal(a, b) for a, b in zip(first, (c.lp, c.ent, c.top_lp)))
    # other logits in the same buffers: nothing is kept
    z2 = logits(rng, 5, 151936)
    c.buf.copy_(torch.from_numpy(z2.astype(np.float32)).reshape(-1))
    c.z = z2.astype(np.float32).astype(np.float64)
    g.replay()
    c.check()


def test_a_model_reads_the_log_probabilities_of_its_last_step():
    from qwen2_decoder_forward_decode_gb300 import DeviceWeights, Model, QwError
    from synth import SHAPES, make_prompt, make_weights
    for name, dt in (("tiny", 0), ("small_bf16", 1)):
        s = SHAPES[name]
        m = Model(s, DeviceWeights(make_weights(s), dt), 32, max_seqs=2)
        try:
            with pytest.raises(QwError):
                m.logprobs([1])  # nothing prefilled
            t = m.prefill(make_prompt(s, 9), seq=1)
            for _ in range(2):
                z = m.logits(seq=1).astype(np.float64)
                lse = z.max() + math.log(np.exp(z - z.max()).sum())
                lp, ranks, ent, top_ids, top_lp = m.logprobs([t, 3], top_k=7, seq=1)
                order = np.lexsort((np.arange(len(z)), -z))
                assert top_ids.tolist() == order[:7].tolist() and top_ids[0] == t and ranks[0] == 1
                np.testing.assert_allclose(lp, z[[t, 3]] - lse, rtol=0, atol=2e-5)
                np.testing.assert_allclose(top_lp, z[order[:7]] - lse, rtol=0, atol=2e-5)
                assert ranks[1] == 1 + int(np.where(order == 3)[0][0])
                p = np.exp(z - lse)
                assert abs(ent + (p * (z - lse)).sum()) < 1e-4
                t = int(m.decode_step()[1])
            for ids, k in (([s.vocab], 0), ([-1], 0), ([0] * 9, 0), ([], 33)):
                with pytest.raises(QwError):
                    m.logprobs(ids, top_k=k, seq=1)
            assert m.position(1) == 11
        finally:
            m.close()


def test_the_first_log_probabilities_of_a_model_do_not_wait_for_the_default_stream():
    """A model with a stream of its own, work pending on the default stream when the scratch is made: the clear must be in
    the model's stream, before the ids and the kernel, and not behind the pending work."""
    from qwen2_decoder_forward_decode_gb300 import DeviceWeights, Model
    from synth import SHAPES, make_prompt, make_weights
    s = SHAPES["tiny"]
    w = DeviceWeights(make_weights(s), 0)
    torch.cuda.synchronize()
    for _ in range(3):
        m = Model(s, w, 32)
        try:
            m.prefill(make_prompt(s, 9))
            z = m.logits().astype(np.float64)
            lse = z.max() + math.log(np.exp(z - z.max()).sum())
            order = np.lexsort((np.arange(len(z)), -z))
            pending = torch.cuda.Event()
            torch.cuda._sleep(10 ** 9)  # about half a second
            pending.record()
            got = m.logprobs([7, 200, 31], top_k=5)
            assert not pending.query(), "the default stream's work was over before the call"
            torch.cuda.synchronize()
            again = m.logprobs([7, 200, 31], top_k=5)
            for lp, ranks, ent, top_ids, top_lp in (got, again):
                np.testing.assert_allclose(lp, z[[7, 200, 31]] - lse, rtol=0, atol=2e-5)
                assert ranks.tolist() == [1 + int(np.where(order == t)[0][0]) for t in (7, 200, 31)]
                assert top_ids.tolist() == order[:5].tolist()
                np.testing.assert_allclose(top_lp, z[order[:5]] - lse, rtol=0, atol=2e-5)
                p = np.exp(z - lse)
                assert abs(ent + (p * (z - lse)).sum()) < 1e-4
        finally:
            m.close()
