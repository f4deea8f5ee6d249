"""The paged-cache operators as they are used together: a decode loop of several sequences that plans
pages, rotates and appends, attends and scores tokens, against a float64 loop over plain arrays."""
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


class Serving:
    """n sequences over one layer's paged cache; the step's projections are given."""

    def __init__(self, n, nq, nkv, hd, page, n_pages, blocks, max_tokens, io, cache, vocab=501):
        from qwen2_decoder_forward_decode_gb300 import binding
        self.b = binding
        self.n, self.nq, self.nkv, self.hd, self.page, self.n_pages, self.blocks, self.max_tokens = n, nq, nkv, hd, page, n_pages, blocks, max_tokens
        self.io, self.cache, self.vocab = io, cache, vocab
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lens, self.new, self.done, self.n_free = i32(n), i32(n), i32(n), torch.tensor([n_pages], dtype=torch.int32, device="cuda")
        self.free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
        self.table, self.cu, self.positions = i32(n, blocks), i32(n + 1), i32(max_tokens)
        self.slots = torch.zeros(max_tokens, dtype=torch.int64, device="cuda")
        self.err = i32(1)
        self.k, self.v = (torch.full((n_pages, nkv, page, hd), float("nan"), dtype=ref.torch_dtype(cache), device="cuda") for _ in range(2))
        self.kv = binding.PagedKV(self.k.data_ptr(), self.v.data_ptr(), ref.CODE[cache], n_pages, page, nkv, hd, nkv * page * hd, page * hd, hd)
        self.turns, self.mscale = binding.rope_turns(hd, 1e4)
        self.freqs = self.turns.astype(np.float64) / 2.0 ** 64 * 2 * math.pi
        self.tturns = torch.from_numpy(self.turns.view(np.int64)).cuda()
        self.qkv = torch.zeros(max_tokens, (nq + 2 * nkv) * hd, dtype=ref.torch_dtype(io), device="cuda")
        self.q = torch.zeros(max_tokens, nq * hd, dtype=ref.torch_dtype(io), device="cuda")
        self.out, self.lse = torch.zeros(n, nq * hd, dtype=ref.torch_dtype(io), device="cuda"), torch.zeros(n, nq, device="cuda")
        self.ws = torch.zeros(binding.paged_attention_workspace(nq, nkv, hd), dtype=torch.uint8, device="cuda")
        self.lws = torch.zeros(binding.token_logprobs_workspace(n, vocab, 3), dtype=torch.uint8, device="cuda")
        self.ids, self.lp, self.ent = i32(n, 1), torch.zeros(n, 1, device="cuda"), torch.zeros(n, device="cuda")
        self.top_ids, self.top_lp = i32(n, 3), torch.zeros(n, 3, device="cuda")
        self.head = torch.randn(nq * hd, vocab, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) / math.sqrt(nq * hd)
        self.logits = torch.zeros(n, vocab, device="cuda")

    def append(self):
        s, p = torch.cuda.current_stream().cuda_stream, lambda t: t.data_ptr()  # noqa: E731
        self.b.page_plan(self.n, self.page, self.n_pages, self.blocks, self.max_tokens, p(self.lens), p(self.new), p(self.free), p(self.n_free), p(self.table), p(self.lens), p(self.n_free),
                         p(self.cu), p(self.positions), p(self.slots), p(self.err), s)
        q, e, row = p(self.qkv), self.qkv.element_size(), self.qkv.shape[1]
        self.b.rope_append(self.kv, self.max_tokens, self.nq, ref.CODE[self.io], p(self.positions), p(self.slots), p(self.tturns), self.hd, False, self.mscale, q, row, q + self.nq * self.hd * e, row,
                           q + (self.nq + self.nkv) * self.hd * e, row, p(self.q), self.nq * self.hd, p(self.err), s)

    def attend(self):
        """One query per sequence: rows 0 .. n - 1 of q (a decode step)."""
        s, p = torch.cuda.current_stream().cuda_stream, lambda t: t.data_ptr()  # noqa: E731
        self.b.paged_attention(self.kv, self.n, self.nq, p(self.table), self.blocks, p(self.lens), ref.CODE[self.io], p(self.q), self.nq * self.hd, 1 / math.sqrt(self.hd), p(self.out),
                               self.nq * self.hd, p(self.lse), p(self.ws), self.ws.numel(), p(self.err), s)
        torch.matmul(self.out.float(), self.head, out=self.logits)
        self.b.token_logprobs(0, self.n, self.vocab, p(self.logits), self.vocab, p(self.ids), 1, p(self.lp), None, p(self.ent), 3, p(self.top_ids), p(self.top_lp), p(self.lws), self.lws.numel(),
                              p(self.err), s)

    def release(self):
        s, p = torch.cuda.current_stream().cuda_stream, lambda t: t.data_ptr()  # noqa: E731
        self.b.page_release(self.n, self.page, self.n_pages, self.blocks, p(self.lens), p(self.done), p(self.table), p(self.free), p(self.n_free), p(self.lens), p(self.n_free), p(self.err), s)


@pytest.mark.parametrize("io,cache,hd,page", [("f32", "f16", 128, 16), ("bf16", "bf16", 64, 7), ("f32", "f32", 16, 1)])
def test_prefill_decode_and_release(io, cache, hd, page):
    n, nq, nkv = 6, 4, 2
    rng = np.random.default_rng(hd)
    s = Serving(n, nq, nkv, hd, page, 6 * ref.pages_of(200, page), ref.pages_of(300, page), 400, io, cache)
    keys, values = [np.zeros((0, nkv, hd)) for _ in range(n)], [np.zeros((0, nkv, hd)) for _ in range(n)]

    def step(new):
        """Appends new[b] tokens to every sequence and mirrors them in the plain arrays."""
        total = sum(new)
        x = torch.from_numpy(rng.standard_normal((total, nq + 2 * nkv, hd))).to(ref.torch_dtype(io))
        s.qkv[:total].copy_(x.reshape(total, -1))
        s.new.copy_(torch.tensor(new, dtype=torch.int32))
        xs = x.double().numpy()
        at, q = 0, []
        for b, add in enumerate(new):
            pos = len(keys[b]) + np.arange(add)
            y = ref.rope(xs[at:at + add, :nq + nkv], pos, s.freqs, False, s.mscale, hd)
            t = lambda a: torch.from_numpy(a).to(ref.torch_dtype(cache)).double().numpy()  # noqa: E731
            keys[b] = np.concatenate([keys[b], t(y[:, nq:])])
            values[b] = np.concatenate([values[b], t(xs[at:at + add, nq + nkv:])])
            q.append(y[:, :nq])
            at += add
        return q

    step([100, 0, 1, 17, 64, 33])
    s.append()
    g = None
    for i in range(8):
        new = [1, 1, 1, 1, 1, 1]
        q = step(new)
        s.ids.copy_(torch.from_numpy(rng.integers(0, s.vocab, (n, 1)).astype(np.int32)))
        if i == 2:  # from here on the step is one graph
            torch.cuda.synchronize()
            lens, n_free = s.lens.clone(), s.n_free.clone()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                s.append()
                s.attend()
            assert torch.equal(s.lens, lens) and torch.equal(s.n_free, n_free)  # (captured, not run)
        if g:
            g.replay()
        else:
            s.append()
            s.attend()
        torch.cuda.synchronize()
        assert int(s.err) == 0
        assert s.lens.tolist() == [len(k) for k in keys]
        out = s.out.double().cpu().numpy().reshape(n, nq, hd)
        for b in range(n):
            for h in range(nkv):
                heads = slice(h * 2, h * 2 + 2)
                o, l, bound = ref.attention(q[b][0, heads], keys[b][:, h], values[b][:, h], 1 / math.sqrt(hd))
                # Rotated queries are rounded to io (one step of it moves a score by 2^-8 or 2^-24 of its
                # size), a key's rounding may fall to the other side of a tie: a step of the cache.
                half = max(ref.EPS_HALF[io], 2 * ref.EPS_HALF[cache] * 0.2, 4 * ref.U)
                wide = 2 * half / math.sqrt(hd) * (np.abs(q[b][0, heads]) @ np.abs(keys[b][:, h]).T).max() * np.abs(values[b][:, h]).max()
                np.testing.assert_array_less(np.abs(out[b, heads] - o), bound + wide + ref.EPS_HALF[io] * np.abs(o) + 1e-9)
        z = s.logits.double().cpu().numpy()
        lse = np.log(np.exp(z - z.max(-1, keepdims=True)).sum(-1)) + z.max(-1)
        ids = s.ids.cpu().numpy()[:, 0]
        np.testing.assert_allclose(s.lp.cpu().numpy()[:, 0], z[np.arange(n), ids] - lse, rtol=0, atol=2e-5)
        np.testing.assert_array_equal(s.top_ids.cpu().numpy(), np.argsort(-z, -1, kind="stable")[:, :3])
        if i == 4:  # two sequences finish and their places start again
            before = int(s.n_free)
            s.done.copy_(torch.tensor([1, 0, 0, 0, 1, 0], dtype=torch.int32))
            s.release()
            back = ref.pages_of(len(keys[0]), page) + ref.pages_of(len(keys[4]), page)
            assert int(s.n_free) == before + back
            for b in (0, 4):
                keys[b], values[b] = np.zeros((0, nkv, hd)), np.zeros((0, nkv, hd))
    # no page in two hands
    used = [int(s.table[b, j]) for b in range(n) for j in range(ref.pages_of(len(keys[b]), page))]
    free = s.free[:int(s.n_free)].tolist()
    assert sorted(used + free) == list(range(s.n_pages))


def test_attention_and_log_probabilities_share_a_workspace_in_turn():
    from qwen2_decoder_forward_decode_gb300 import binding
    s = Serving(5, 4, 2, 64, 16, 200, 40, 3000, "f32", "f16")
    s.new.copy_(torch.tensor([600, 1, 0, 33, 500], dtype=torch.int32))
    s.qkv.normal_(generator=torch.Generator("cuda").manual_seed(2))
    s.append()
    s.attend()
    torch.cuda.synchronize()
    want = [t.clone() for t in (s.out, s.lse, s.lp, s.ent, s.top_ids)]
    n = max(s.ws.numel(), s.lws.numel())
    s.ws = s.lws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for t in (s.out, s.lse, s.lp, s.ent, s.top_ids):
            t.zero_()
        s.attend()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (s.out, s.lse, s.lp, s.ent, s.top_ids)))
    assert int(s.err) == 0 and binding.DEV_PAGE == 32
