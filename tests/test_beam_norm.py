"""The normaliser of beam selection: next to 64 bits where few tokens carry a row, where a row's logits lie near the border of the
plain range, and between rows that differ by a constant."""
import math

import numpy as np
import pytest

import paged_ref as ref
from test_beam_select import Call, rand_logits

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def log_probs(z):
    """Largest logit's log probability [rows] and the mass [rows] of tokens below 2^-10 of a row's sum."""
    top = z.max(-1, keepdims=True)
    e = np.exp(z - top)
    s = e.sum(-1, keepdims=True)
    return -np.log(s)[:, 0], (np.where(e < 1.01 * 2.0 ** -10 * s, e, 0).sum(-1, keepdims=True) / s)[:, 0]


KINDS = ["certain", "two", "neighbours", "fifty", "lowest", "five hundred", "falling", "rising", "bulk"]


def make(kind, rows, vocab, dtype):
    z = rand_logits(rows, vocab, dtype, 11).double()
    gen = torch.Generator().manual_seed(3)
    pick = torch.randperm(vocab, generator=gen)
    if kind == "certain":
        z[:, pick[0]] = 30.0 + torch.arange(rows).double() / 3
    if kind == "two":
        z[:, pick[0]], z[:, pick[1]] = 30.3, 29.7
    if kind == "neighbours":  # in one lane's registers
        at = vocab // 2 // 8 * 8
        z[:, at:at + 8] = 28 + torch.randn(rows, len(z[0, at:at + 8]), generator=gen).double()
    if kind in ("fifty", "lowest", "five hundred"):
        n = min(500 if kind == "five hundred" else 50, vocab)
        left = z[:, pick[:n]].clone() if kind != "five hundred" else 0.4 * torch.rand(rows, n, generator=gen).double()
        z[:] = torch.finfo(ref.torch_dtype(dtype)).min if kind == "lowest" else -INF
        z[:, pick[:n]] = left
    if kind in ("falling", "rising"):  # every chunk moves the reference, or none after the first
        z += torch.linspace(40, -40, vocab).double() * (1 if kind == "falling" else -1)
    return z.to(ref.torch_dtype(dtype))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vocab,rows,gap", [(100, 6, 0), (5003, 6, 0), (5003, 6, 1), (152064, 6, 0), (20011, 700, 0)])
def test_normalisers_are_near_64_bits(dtype, kind, vocab, rows, gap):
    z = make(kind, rows, vocab, dtype)
    lp, light = log_probs(z.double().numpy())
    scores = (-lp).astype(np.float32)  # the best candidate's score is then near 0, where fp32 shows the normaliser's own error
    c = Call(z, 1, 1, scores, gap=gap)
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    want = scores.astype(np.float64) + lp
    got = c.scores_out[:rows].double().cpu().numpy()
    # tokens above 2^-10 of the sum are taken in 64 bits. The others' exponentials are good to 2^-22, their exponents of up to 32
    # binary places to 2^-20 ln 2, and sums of some of them to 2^-23: less than 2^-19 of their mass. The 512 numbers of a piece's
    # lanes are rounded to 2^-39 of at most twice the sum, less than 2^-29.
    tol = light * 2.0 ** -19 + 2.0 ** -29 + 2.0 ** -24 * np.abs(want)
    np.testing.assert_array_less(np.abs(got - want), tol)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [3000, 152064])
def test_a_likely_token_costs_next_to_nothing(dtype, vocab):
    """Probabilities next to 1: their logarithm is negative, and near that of 64 bits relative to its own size."""
    z = rand_logits(8, vocab, dtype, 5, 1.0).double()
    z[:, 1234] = torch.linspace(18, 32, 8).double()
    z = z.to(ref.torch_dtype(dtype))
    lp, _ = log_probs(z.double().numpy())
    c = Call(z, 1, 1, [0.0] * 8)
    c.run()
    torch.cuda.synchronize()
    got = c.scores_out[:8].double().cpu().numpy()
    assert (got < 0).all()
    # (everything but one token is light: 2^-19 of the rest, the sum's 2^-29 as above)
    np.testing.assert_array_less(np.abs(got - lp), 2.0 ** -18 * np.abs(lp) + 2.0 ** -29)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [700, 152064])
@pytest.mark.parametrize("left", [1, 2, 40])
def test_rows_that_differ_by_a_constant_tie(dtype, vocab, left):
    """Few tokens allowed, all scores equal: by definition the beams' candidates tie, and the lower beam comes first."""
    gen = torch.Generator().manual_seed(left)
    at = torch.randperm(vocab, generator=gen)[:left]
    base = torch.randint(-16, 17, (left,), generator=gen) / 8
    z = torch.full((8, vocab), -INF)
    for row, shift in enumerate([3.0, 0.375, -2.125, 7.5, -6.625, 0.0, 5.25, -0.875]):
        z[row, at] = base + shift
    c = Call(z.to(ref.torch_dtype(dtype)), 8, 8, [-1.25] * 8)
    c.run()
    torch.cuda.synchronize()
    best = sorted(at[base == base.max()].tolist())
    assert list(zip(c.parents[:8].tolist(), c.tokens[:8].tolist())) == [(row, t) for row in range(8) for t in best][:8]
    lp = -math.log(float(torch.exp(base.double() - base.double().max()).sum()))
    assert set(c.scores_out[:8].tolist()) == {float(np.float32(-1.25 + lp))} if left == 1 else len(set(c.scores_out[:8].tolist())) == 1
    assert abs(float(c.scores_out[0]) - (-1.25 + lp)) <= 2.0 ** -24 * abs(-1.25 + lp) + 2.0 ** -29


@pytest.mark.parametrize("vocab", [600, 8192, 70000])
def test_rows_across_the_border_of_far_logits(vocab):
    far = 2.0 ** 20
    gen = torch.Generator().manual_seed(vocab)
    z = torch.full((10, vocab), -far)
    z[0, 77] = -far + 0.0625
    z[1, vocab - 1] = -far + 0.5
    z[2] += torch.randint(-8, 9, (vocab,), generator=gen) / 8
    z[3] += torch.randint(-800, 801, (vocab,), generator=gen) / 8
    z[4, ::3] = -far + 40.0
    z[5, 300:] = -far - 3.0
    z[6] = far - 0.0625 * torch.randint(0, 30, (vocab,), generator=gen)
    z[7] = far + torch.randint(-30, 31, (vocab,), generator=gen) / 8
    z[8, 5] = -far + 200.0
    z[9, :500] = -far + 127.0
    c = Call(z, 1, 4, [-1.0] * 10)
    c.run()
    c.check()
    assert int(c.err) == 0
