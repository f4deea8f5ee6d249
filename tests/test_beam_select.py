"""Beam selection on the GPU against the definition in 64 bits."""
import math

import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Call:
    def __init__(self, logits, beams, n_out, scores, ended=None, weights=None, end_id=-1, width=0, gap=0, offset=0, seed=0, ended_out=True):
        """logits: a float torch tensor [rows][vocab]; gap elements between rows, offset before the first."""
        from qwen2_decoder_forward_decode_gb300 import binding
        self.rows, self.vocab = logits.shape
        self.beams, self.n_out, self.end_id, self.width = beams, n_out, end_id, width
        self.groups = self.rows // beams
        self.dtype = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[logits.dtype]
        self.z = logits.double().numpy()
        self.stride = self.vocab + gap
        buf = torch.full((offset + self.rows * self.stride,), float("nan"), dtype=logits.dtype)
        buf[offset:].view(self.rows, self.stride)[:, :self.vocab] = logits
        self.buf = buf.cuda()
        self.ptr = self.buf.data_ptr() + offset * self.buf.element_size()
        f32 = lambda a: torch.tensor(np.asarray(a, dtype=np.float32)).cuda()  # noqa: E731
        i32 = lambda a: torch.tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.scores, self.tscores = np.asarray(scores, dtype=np.float32).astype(np.float64), f32(scores)
        self.ended, self.tended = np.zeros(self.rows, dtype=bool) if ended is None else np.asarray(ended).astype(bool), None if ended is None else i32(ended)
        self.weights, self.tweights = np.ones(self.rows) if weights is None else np.asarray(weights, dtype=np.float32).astype(np.float64), None if weights is None else f32(weights)
        k = self.groups * n_out
        rng = np.random.default_rng(seed)
        self.lens, self.history = rng.integers(0, max(width, 1), self.rows), rng.integers(0, 1000, (self.rows, max(width, 1)))
        self.tlens, self.thistory = i32(self.lens), i32(self.history)
        full = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
        self.parents, self.tokens, self.lens_out, self.history_out = full(k + 2), full(k + 2), full(k + 2), full(k + 1, max(width, 1))
        self.ended_out = full(k + 2) if ended_out else None
        self.scores_out = torch.full((k + 2,), 77.0, device="cuda")
        self.ws = torch.full((binding.beam_select_workspace(self.groups, beams, self.vocab, n_out),), 0x5a, dtype=torch.uint8, device="cuda")  # (need not be zeroed)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self):
        from qwen2_decoder_forward_decode_gb300 import binding
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        w = self.width > 0
        binding.beam_select(ref.CODE[self.dtype], self.groups, self.beams, self.vocab, self.ptr, self.stride, p(self.tscores), p(self.tweights), p(self.tended), self.end_id, self.n_out,
                            p(self.parents), p(self.tokens), p(self.scores_out), p(self.ended_out), self.width, p(self.thistory) if w else None, p(self.tlens) if w else None,
                            p(self.history_out) if w else None, p(self.lens_out) if w else None, p(self.ws), self.ws.numel(), p(self.err), torch.cuda.current_stream().cuda_stream)

    def want(self):
        """[(parent, token, score, ended)] of every group, and the rows without a distribution."""
        out, bad = [], []
        for g in range(self.groups):
            found = []
            for w in range(g * self.beams, (g + 1) * self.beams):
                c, z = self.scores[w], self.z[w]
                if math.isnan(c) or c == INF or not 0 < self.weights[w] < INF:
                    bad.append(w)
                    continue
                if c == -INF:
                    continue
                if self.ended[w]:
                    found.append((-self.weights[w] * c, w, 0, self.end_id, c, True))
                    continue
                top = z.max()
                if math.isnan(z.sum()) or top == INF or top == -INF:
                    bad.append(w)
                    continue
                norm = top + math.log(np.exp(z - top).sum())
                order = np.lexsort((np.arange(self.vocab), -z))[:self.n_out]
                for t in order[z[order] > -INF].tolist():
                    s = c + (z[t] - norm)
                    found.append((-self.weights[w] * s, w, -z[t], t, s, t == self.end_id))
            found.sort(key=lambda f: f[:4])
            out.append([(f[1], f[3], f[4], f[5]) for f in found[:self.n_out]])
        return out, bad

    def check(self):
        torch.cuda.synchronize()
        want, bad = self.want()
        assert bool(int(self.err) & 2) == bool(bad)
        k = self.groups * self.n_out
        parents, tokens, scores = self.parents.tolist(), self.tokens.tolist(), self.scores_out.double().tolist()
        ended = self.ended_out.tolist() if self.ended_out is not None else None
        lens, history = self.lens_out.tolist(), self.history_out.cpu().numpy()
        assert parents[k:] == tokens[k:] == [-77] * 2 and scores[k:] == [77.0] * 2 and (history[k:] == -77).all()
        for g in range(self.groups):
            rows = want[g] + [(-1, -1, -INF, True)] * (self.n_out - len(want[g]))
            at = slice(g * self.n_out, (g + 1) * self.n_out)
            assert parents[at] == [r[0] for r in rows], g
            assert tokens[at] == [r[1] for r in rows], g
            if ended:
                assert ended[at] == [int(r[3]) for r in rows]
            for i, (parent, token, score, _) in enumerate(rows):
                got = scores[g * self.n_out + i]
                # half a step of the rounded score; the normaliser: each exponential is good to 2^-22 (ex2), its exponent of up to 8
                # binary places weighs as much again where it counts, and a weighted mean of relative errors is no larger
                assert got == score or abs(got - score) <= 2.0 ** -24 * abs(score) + 2.0 ** -21, (g, i, got, score)
                if not self.width:
                    continue
                o = g * self.n_out + i
                line = [] if parent < 0 else self.history[parent, :self.lens[parent]].tolist() + ([] if self.ended[parent] else [token])
                assert lens[o] == len(line) and history[o, :len(line)].tolist() == line and (history[o, len(line):] == -77).all()


def rand_logits(rows, vocab, dtype, seed=0, scale=3.0):
    return (scale * torch.randn(rows, vocab, generator=torch.Generator().manual_seed(seed))).to(ref.torch_dtype(dtype))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("groups,beams,vocab,n_out", [
    (1, 1, 1, 1), (1, 2, 1, 4), (3, 2, 5, 8), (2, 4, 100, 8), (1, 1, 255, 32), (1, 3, 257, 32), (5, 4, 1000, 4), (2, 32, 3000, 32), (1, 4, 151936, 8), (3, 5, 32001, 10), (20, 4, 20011, 8), (1, 32, 70000, 32),
    (1, 1, 500000, 32), (1, 2, 2097152, 5),
])
def test_candidates_match_the_definition(dtype, groups, beams, vocab, n_out):
    rng = np.random.default_rng(vocab + beams)
    c = Call(rand_logits(groups * beams, vocab, dtype, vocab), beams, n_out, -10 * rng.random(groups * beams), width=9)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gap,offset", [(0, 1), (1, 0), (3, 5), (8, 8)])
def test_strided_and_misaligned_rows(dtype, gap, offset):
    c = Call(rand_logits(6, 5003, dtype), 3, 6, [-1, -2, -3, -1.5, -1.25, -1], gap=gap, offset=offset)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ended_and_absent_beams(dtype):
    z = rand_logits(12, 700, dtype)
    z[1] = float("nan")  # of an ended beam: not looked at
    z[6] = -INF          # of an absent one
    scores = [-3, -2, -9, -1, -INF, -4, -INF, -INF, -INF, -INF, -0.5, -30]
    c = Call(z, 4, 6, scores, ended=[0, 1, 0, 1, 0, 0, 0, 0, 1, 1, 1, 1], end_id=17, width=5)
    c.run()
    c.check()
    assert int(c.err) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_weights_rank_by_length(dtype):
    rng = np.random.default_rng(2)
    z = rand_logits(24, 3001, dtype)
    z[:, 5] = 12.0
    c = Call(z, 4, 8, -20 * rng.random(24), ended=rng.random(24) < 0.3, weights=1 / rng.integers(1, 40, 24) ** 0.6, end_id=5, width=40)
    c.run()
    c.check()


def test_the_first_step_of_equal_beams():
    """Equal rows give equal scores, and the lower beam comes first; at the very first step all but one beam are absent."""
    z = rand_logits(1, 9000, "f32").repeat(8, 1)
    for scores in ([0.0] + [-INF] * 3 + [-1.0] * 4, [-2.0] * 8):
        c = Call(z, 4, 8, scores)
        c.run()
        c.check()
    c = Call(z, 4, 8, [-2.0] * 8, gap=1)  # rows on different boundaries are summed alike
    c.run()
    c.check()
    assert c.parents[:4].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["constant", "steps", "masked", "lowest", "few", "last", "signed zeros", "descending", "infinite", "one"])
def test_ties_and_masks(dtype, kind):
    vocab, t = 40000, ref.torch_dtype(dtype)
    z = rand_logits(4, vocab, dtype, 7)
    low = torch.finfo(t).min
    if kind == "constant":
        z[:] = 2.5
    if kind == "steps":
        z = (z / 2).round() * 2
    if kind == "masked":
        z[:, torch.rand(vocab, generator=torch.Generator().manual_seed(1)) < 0.99] = -INF
    if kind == "lowest":  # nothing is left: all tokens are as likely
        z[0] = low
        z[1] = low
        z[1, 777] = 3.0
    if kind == "few":  # three tokens above the mask, the rest of the candidates from the masked ones
        z[:] = low
        z[:, [39999, 5, 20000]] = torch.tensor([1.0, 0.5, 0.25]).to(t)
    if kind == "last":
        z[:, -3:] = 30.0
    if kind == "signed zeros":
        z = torch.zeros(4, vocab, dtype=t)
        z[:, ::2] = -0.0
    if kind == "descending":
        z = torch.linspace(8, -8, vocab).repeat(4, 1).to(t)
    if kind == "infinite":  # three tokens only
        z[:] = -INF
        z[:, [39999, 5, 20000]] = torch.tensor([1.0, 0.5, 0.25]).to(t)
    if kind == "one":
        z[:] = -INF
        z[:, 12345] = -3.0
    c = Call(z, 2, 16, [-1.0, -1.5, -7.0, -0.25])
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_and_far_logits(dtype):
    z = rand_logits(8, 3000, dtype)
    z[1] *= 1e5
    z[2] = z[2] * 1e30
    z[3] += 1e4
    z[4] -= 2e6
    z[5] = torch.finfo(z.dtype).max * torch.sign(z[5].float()).to(z.dtype)
    z[6] *= 1e-30
    z[7, 11] = torch.finfo(z.dtype).max
    c = Call(z, 1, 5, [-1.0] * 8)
    c.run()
    c.check()


def test_rows_without_a_distribution():
    z = rand_logits(8, 2000, "f32")
    z[0, 1999] = float("nan")
    z[1, 3] = INF
    z[2] = -INF
    scores = [-1.0, -1.0, -1.0, -2.0, float("nan"), INF, -1.0, -1.0]
    weights = [1, 1, 1, 1, 1, 1, 0, 0.5]
    c = Call(z, 4, 8, scores, weights=weights)
    c.run()
    c.check()
    assert int(c.err) == 2
    for bad in (-1.0, float("nan"), INF):
        c = Call(z[3:4], 1, 2, [-1.0], weights=[bad])
        c.run()
        c.check()
        assert int(c.err) == 2 and c.parents[:2].tolist() == [-1, -1]


def test_full_histories_are_reported():
    c = Call(rand_logits(2, 50, "f32"), 2, 2, [-1.0, -1.1], width=4)
    c.tlens.copy_(torch.tensor([4, 4], dtype=torch.int32))
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == 64 and c.lens_out[:2].tolist() == [4, 4]
    for i in range(2):
        assert c.history_out[i].tolist() == c.thistory[c.parents[i]].tolist()
    c = Call(rand_logits(2, 50, "f32"), 2, 2, [-1.0, -1.1], width=4)
    c.tlens.copy_(torch.tensor([-1, 9], dtype=torch.int32))
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == 64


def test_scores_lie_closer_than_fp32_tells():
    """Two beams whose candidates differ by 4e-7 at scores near -1000, where fp32 has steps of 6e-5: the order is that of the
    scores before they are rounded."""
    z = torch.zeros(2, 1000)
    z[0, 500], z[1, 400] = 5.0, 5.0 + 4.8e-7
    for scores, first in (([-1000.0, -1000.0], 1),):
        c = Call(z, 2, 2, scores)
        c.run()
        c.check()
        assert c.parents[0] == first


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_bit_by_bit_captured_and_on_another_stream(dtype):
    c = Call(rand_logits(12, 30011, dtype), 4, 8, -5 * np.random.default_rng(0).random(12), ended_out=False, width=6)
    c.run()
    c.check()
    want = [t.clone() for t in (c.parents, c.tokens, c.scores_out, c.history_out)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for i in range(4):
        c.scores_out.zero_()
        c.ws.fill_(0xff)
        torch.cuda.synchronize()
        if i % 2:
            g.replay()
        else:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                c.scores_out.fill_(77.0)
                c.run()
            s.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(c.scores_out[:24], want[2][:24]) and all(torch.equal(a, b) for a, b in zip((c.parents, c.tokens, c.history_out), (want[0], want[1], want[3])))


def test_many_groups():
    rng = np.random.default_rng(9)
    c = Call(rand_logits(3000, 300, "f16"), 2, 4, -3 * rng.random(3000), ended=rng.random(3000) < 0.1, end_id=0)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gap", [0, 1])
@pytest.mark.parametrize("vocab", [100, 2000, 33000])
def test_a_nan_anywhere_leaves_a_row_without_candidates(dtype, gap, vocab):
    z = rand_logits(6, vocab, dtype, 3)
    for row, at in enumerate((0, vocab - 1, vocab // 2, vocab // 3, 7)):
        z[row, at] = float("nan")
    z[1, vocab - 1] = -float("nan")
    c = Call(z, 3, 4, [-1.0] * 6, gap=gap)
    c.run()
    c.check()
    assert int(c.err) == 2 and c.parents[4:8].tolist() == [5] * 4


def test_two_streams_with_their_own_workspaces():
    calls = [Call(rand_logits(16, 40000, "bf16", i), 4, 8, -np.random.default_rng(i).random(16), width=30, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    for c in calls:
        c.check()
