"""Shared attention of 16-bit callers: probabilities keep two pieces of the cache's type, over shared and own positions alike."""
import numpy as np
import pytest

import paged_ref as ref
from test_shared_attention import Call

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("cache", ["f16", "bf16"])
@pytest.mark.parametrize("groups,nq,nkv,hd,page,q_scale", [
    ([(200, [201, 210, 200])], 8, 2, 128, 16, 2.0), ([(700, [700 + i for i in range(40)])], 8, 2, 64, 16, 1.0), ([(4000, [4001] * 20), (100, [150])], 28, 4, 128, 64, 0.5),
    ([(130, [131, 140])] * 5, 12, 2, 32, 5, 2.0), ([(1500, [1500])], 4, 4, 96, 8, 8.0), ([(16383, [16384] * 33)], 8, 1, 128, 16, 1.0),
])
@pytest.mark.parametrize("scale", [None, -0.07])
def test_probabilities_keep_two_pieces(cache, groups, nq, nkv, hd, page, q_scale, scale):
    c = Call(groups, nq, nkv, hd, page, cache, cache, q_scale=q_scale, scale=scale)
    c.run()
    got, _ = c.got()
    assert int(c.err) == 0
    q = c.tq.double().cpu().numpy()[:len(c.lens), :nq * hd].reshape(got.shape)
    g = nq // nkv
    piece = ref.EPS_HALF[cache] ** 2  # what the second piece's rounding leaves
    for b, n in enumerate(c.lens):
        for h in range(nkv):
            heads = slice(h * g, (h + 1) * g)
            k, v = c.c.k[b][:n, h], c.c.v[b][:n, h]
            o, _, bound = ref.attention(q[b, heads], k, v, c.scale)
            z = c.scale * (q[b, heads] @ k.T)
            p = np.exp(z - z.max(-1, keepdims=True))
            bound = bound + piece * (p / p.sum(-1, keepdims=True)) @ np.abs(v)
            if cache == "f16":  # times 2^10: half a step of the smallest numbers is 2^-35 of the largest probability
                bound = bound + 2.0 ** -35 / p.sum(-1, keepdims=True) * np.abs(v).sum(0)
            tol = bound + ref.EPS_HALF[cache] * (np.abs(o) + bound) + ref.TINY[cache]
            np.testing.assert_array_less(np.abs(got[b, heads] - o), tol, err_msg=f"sequence {b} KV head {h}")
