"""The normaliser of beam selection where a row's logits lie near the border of the plain range."""
import pytest

from test_beam_select import Call

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


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
