"""The operators for continuations of a prompt as they are used together: a beam search over a paged cache that
plans, appends, attends over the shared prompt, selects, forks, copies and now and then compacts, against plain
float64 arrays that hold every beam by itself."""
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


class Search:
    """G prompts of W beams over one layer; a token's query, key and value are rows of given tables."""

    def __init__(self, G, W, nq, nkv, hd, page, n_pages, blocks, vocab, io, cache, width):
        from qwen2_decoder_forward_decode_gb300 import binding
        self.b = binding
        self.G, self.W, self.n, self.nq, self.nkv, self.hd, self.page, self.n_pages, self.blocks, self.vocab, self.width = G, W, G * W, nq, nkv, hd, page, n_pages, blocks, vocab, width
        self.io, self.cache = io, cache
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        n = self.n
        self.lens, self.lens2, self.table, self.table2 = i32(n), i32(n), i32(n, blocks), i32(n, blocks)
        self.shares, self.free, self.n_free = i32(n_pages), torch.arange(n_pages, dtype=torch.int32, device="cuda"), torch.full((1,), n_pages, dtype=torch.int32, device="cuda")
        self.new, self.cu, self.positions, self.slots = i32(n), i32(n + 1), i32(4096), torch.zeros(4096, dtype=torch.int64, device="cuda")
        self.src, self.dst, self.count = i32(n), i32(n), i32(n)
        self.mv_src, self.mv_dst, self.n_moves = i32(64), i32(64), i32(1)
        self.err = i32(1)
        # two layers' caches: the second holds what the first does, doubled, so that copies reach all layers
        self.kv = [[torch.full((n_pages, nkv, page, hd), float("nan"), dtype=ref.torch_dtype(cache), device="cuda") for _ in range(2)] for _ in range(2)]
        self.pk = [binding.PagedKV(k.data_ptr(), v.data_ptr(), ref.CODE[cache], n_pages, page, nkv, hd, nkv * page * hd, page * hd, hd) for k, v in self.kv]
        self.pks = binding.paged_kv_array(self.pk)
        self.turns, self.mscale = binding.rope_turns(hd, 1e4)
        self.freqs = self.turns.astype(np.float64) / 2.0 ** 64 * 2 * math.pi
        self.tturns = torch.from_numpy(self.turns.view(np.int64)).cuda()
        rng = np.random.default_rng(3)
        self.tokens_qkv = torch.from_numpy(rng.standard_normal((vocab, (nq + 2 * nkv) * hd))).to(ref.torch_dtype(io))
        self.ttokens = self.tokens_qkv.cuda()
        self.head = torch.from_numpy(rng.standard_normal((nq * hd, vocab)) * 6 / math.sqrt(nq * hd)).float()
        self.thead = self.head.cuda()
        self.group_cu = torch.arange(0, n + 1, W, dtype=torch.int32, device="cuda")
        self.shared = i32(n)
        self.q = torch.zeros(4096, nq * hd, dtype=ref.torch_dtype(io), device="cuda")
        self.out = torch.zeros(n, nq * hd, dtype=ref.torch_dtype(io), device="cuda")
        self.logits = torch.zeros(n, vocab, device="cuda")
        self.scores, self.scores2 = torch.full((n,), -math.inf, device="cuda"), torch.zeros(n, device="cuda")
        self.ended, self.ended2, self.parents, self.tokens = i32(n), i32(n), i32(n), i32(n)
        self.history, self.history2, self.hlens, self.hlens2 = i32(n, width), i32(n, width), i32(n), i32(n)
        w = lambda size: torch.zeros(size, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws_attn, self.ws_beam = w(binding.shared_attention_workspace(n, nq, nkv, hd)), w(binding.beam_select_workspace(G, W, vocab, W))
        self.ws_fork, self.ws_pack = w(binding.page_fork_workspace(n_pages)), w(binding.page_compact_workspace(n_pages))

    def p(self, *names):
        return [getattr(self, x).data_ptr() for x in names]

    def append(self, ids, max_tokens):
        """One token of ids [max_tokens] (device) for every place that the plan hands out."""
        s = torch.cuda.current_stream().cuda_stream
        self.b.page_plan(self.n, self.page, self.n_pages, self.blocks, max_tokens, *self.p("lens", "new", "free", "n_free", "table", "lens", "n_free", "cu", "positions", "slots", "err"), s)
        x = self.ttokens[ids.long()].contiguous()
        row, e, q = x.shape[1], x.element_size(), x.data_ptr()
        for layer in range(2):
            if layer:
                x = x.clone()
                x[:, self.nq * self.hd:] *= 2
                q = x.data_ptr()
            self.b.rope_append(self.pk[layer], max_tokens, self.nq, ref.CODE[self.io], *self.p("positions", "slots", "tturns"), self.hd, False, self.mscale, q, row, q + self.nq * self.hd * e, row,
                               q + (self.nq + self.nkv) * self.hd * e, row, self.q.data_ptr(), self.nq * self.hd, self.err.data_ptr(), s)
        self.keep = x

    def attend(self):
        s = torch.cuda.current_stream().cuda_stream
        self.b.shared_attention(self.pk[0], self.n, self.nq, self.table.data_ptr(), self.blocks, self.lens.data_ptr(), self.G, *self.p("group_cu", "shared"), ref.CODE[self.io], self.q.data_ptr(),
                                self.nq * self.hd, 1 / math.sqrt(self.hd), self.out.data_ptr(), self.nq * self.hd, None, self.ws_attn.data_ptr(), self.ws_attn.numel(), self.err.data_ptr(), s)
        torch.matmul(self.out.float(), self.thead, out=self.logits)

    def select(self, end):
        s = torch.cuda.current_stream().cuda_stream
        self.b.beam_select(0, self.G, self.W, self.vocab, self.logits.data_ptr(), self.vocab, self.scores.data_ptr(), None, self.ended.data_ptr(), end, self.W,
                           *self.p("parents", "tokens", "scores2", "ended2"), self.width, *self.p("history", "hlens", "history2", "hlens2", "ws_beam"), self.ws_beam.numel(), self.err.data_ptr(), s)
        for a in ("scores", "ended", "history", "hlens"):
            x, y = getattr(self, a), getattr(self, a + "2")
            setattr(self, a, y)
            setattr(self, a + "2", x)

    def fork(self):
        s = torch.cuda.current_stream().cuda_stream
        self.b.page_fork(self.n, self.n, self.page, self.n_pages, self.blocks, *self.p("lens", "table", "parents", "shares", "free", "n_free", "lens2", "table2", "shares", "free", "n_free", "src",
                                                                                     "dst", "count", "ws_fork"), self.ws_fork.numel(), self.err.data_ptr(), s)
        self.b.page_copy(self.pks, 2, self.n, *self.p("src", "dst", "count", "err"), s)
        self.lens, self.lens2, self.table, self.table2 = self.lens2, self.lens, self.table2, self.table

    def compact(self):
        s = torch.cuda.current_stream().cuda_stream
        self.b.page_compact(self.n, self.page, self.n_pages, self.blocks, 64, *self.p("lens", "table", "shares", "free", "n_free", "table", "shares", "free", "mv_src", "mv_dst", "n_moves", "ws_pack"),
                            self.ws_pack.numel(), self.err.data_ptr(), s)
        self.b.page_copy(self.pks, 2, 64, *self.p("mv_src", "mv_dst"), None, self.err.data_ptr(), s)

    def check_pool(self):
        torch.cuda.synchronize()
        assert int(self.err) == 0
        held = np.zeros(self.n_pages, dtype=int)
        lens, table = self.lens.tolist(), self.table.cpu().numpy()
        for b, n in enumerate(lens):
            np.add.at(held, table[b, :ref.pages_of(n, self.page)], 1)
        free = self.free[:int(self.n_free)].tolist()
        assert sorted(free) == np.flatnonzero(held == 0).tolist()
        np.testing.assert_array_equal(self.shares.cpu().numpy(), np.maximum(held - 1, 0))

    def rows(self, b, layer):
        """Keys and values [len][nkv][hd] of sequence b."""
        n, t = int(self.lens[b]), self.table[b].long()
        at = torch.arange(n, device="cuda")
        return [c[t[at // self.page], :, at % self.page].double().cpu().numpy() for c in self.kv[layer]]


@pytest.mark.parametrize("io,cache,nq,nkv,hd,page", [("f32", "f16", 4, 2, 64, 8), ("bf16", "bf16", 14, 2, 128, 16), ("f32", "f32", 4, 1, 32, 5), ("f32", "bf16", 6, 3, 64, 1)])
def test_a_beam_search_over_pages(io, cache, nq, nkv, hd, page):
    G, W, vocab, end, steps = 3, 4, 61, 7, 24
    prompts = [90, 33, 128]
    rng = np.random.default_rng(hd + page)
    s = Search(G, W, nq, nkv, hd, page, G * ref.pages_of(130, page) + G * W * (2 + ref.pages_of(steps + 2, page)), ref.pages_of(160, page), vocab, io, cache, 40)
    # the prompts go into each group's first beam, their last token's logits start the search
    ids = [rng.integers(0, vocab, n) for n in prompts]
    text = {g * W: list(ids[g]) for g in range(G)}
    s.new.zero_()
    s.new[::W] = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    total = sum(prompts)
    s.append(torch.from_numpy(np.concatenate(ids)).cuda(), total)
    s.shared.copy_(torch.tensor(np.repeat(prompts, W), dtype=torch.int32))
    last = torch.cumsum(torch.tensor(prompts), 0).cuda() - 1
    first_q = s.q[last].clone()
    s.q[:s.n].zero_()
    s.q[0:s.n:W] = first_q
    s.scores[::W] = 0.0
    beams = [list(text[b]) if b % W == 0 else None for b in range(s.n)]  # tokens of every beam, the prompt's among them
    scores, ended = np.where(np.arange(s.n) % W == 0, 0.0, -np.inf), np.zeros(s.n, dtype=bool)
    kv_of = lambda x: ref.torch_dtype(cache)  # noqa: E731

    def plain_logits(tokens):
        """The search's logits for one beam: all keys and values again, in 64 bits from what the cache rounds to."""
        x = s.tokens_qkv[tokens].double().numpy().reshape(len(tokens), nq + 2 * nkv, hd)
        y = ref.rope(x[:, :nq + nkv], np.arange(len(tokens)), s.freqs, False, s.mscale, hd)
        r = lambda a: torch.from_numpy(a).to(kv_of(0)).double().numpy()  # noqa: E731
        k, v, q = r(y[:, nq:]), r(x[:, nq + nkv:]), torch.from_numpy(y[-1, :nq]).to(ref.torch_dtype(io)).double().numpy()
        g = nq // nkv
        out = np.concatenate([ref.attention(q[h * g:(h + 1) * g], k[:, h], v[:, h], 1 / math.sqrt(hd))[0] for h in range(nkv)])
        return out.reshape(-1) @ s.head.double().numpy()

    for step in range(steps):
        s.attend()
        s.select(end)
        torch.cuda.synchronize()
        assert int(s.err) == 0
        parents, tokens, got, got_ended = s.parents.tolist(), s.tokens.tolist(), s.scores.double().tolist(), s.ended.tolist()
        # A logit is a sum of nq hd outputs times weights of deviation 6 / sqrt(nq hd): its error's deviation is 6 times an
        # output's. bf16: 2^-8 of rounding and as much again of probabilities, outputs of at most about one: 6 sqrt(2) 2^-8 =
        # 0.033, times 4.5 for the worst of some thousand. fp32: 2^-18 there, and a key that rounds to the cache's other
        # neighbour where 64 bits and 32 differ (one in thousands): 2^-8 of one product of hd, a tenth of a logit's step at most.
        tol = {"f32": 2e-3, "bf16": 0.15}[io]
        new_beams, new_scores, new_ended = [], [], []
        for g in range(G):
            found = {}
            for w in range(g * W, (g + 1) * W):
                if scores[w] == -np.inf:
                    continue
                if ended[w]:
                    found[(w, end)] = scores[w]
                    continue
                z = plain_logits(beams[w])
                z = z - z.max()
                lp = z - math.log(np.exp(z).sum())
                for t in range(vocab):
                    found[(w, t)] = scores[w] + lp[t]
            best = sorted(found.values(), reverse=True)[:W]
            picked = set()
            for i in range(g * W, (g + 1) * W):
                key = (parents[i], tokens[i])
                assert key in found and key not in picked, (step, i, key)
                picked.add(key)
                # the score, and a place among the best (candidates closer than the tolerance may change places)
                assert abs(found[key] - got[i]) <= tol and abs(found[key] - best[i - g * W]) <= 2 * tol, (step, i, key, found[key], got[i], best)
                old = bool(ended[parents[i]])
                assert bool(got_ended[i]) == (old or tokens[i] == end)
                new_beams.append(beams[parents[i]] + ([] if old else [tokens[i]]))
                new_scores.append(got[i])
                new_ended.append(bool(got_ended[i]))
        beams, scores, ended = new_beams, np.array(new_scores), np.array(new_ended)
        s.fork()
        if step % 5 == 3:
            s.compact()
        s.check_pool()
        # the tokens chosen go in; an ended beam gets no position
        s.new.copy_(torch.tensor([0 if e else 1 for e in ended], dtype=torch.int32))
        live = [b for b in range(s.n) if not ended[b]]
        feed = torch.zeros(s.n, dtype=torch.int64, device="cuda")
        feed[:len(live)] = torch.tensor([beams[b][-1] for b in live], device="cuda")
        s.append(feed, s.n)
        q = torch.zeros_like(s.q[:s.n])
        if live:
            q[torch.tensor(live, device="cuda")] = s.q[:len(live)]
        s.q[:s.n] = q
        s.check_pool()
        for b in range(s.n):
            assert s.history[b, :int(s.hlens[b])].tolist() == beams[b][prompts[b // W]:]
            held = beams[b] if not ended[b] else beams[b][:-1]  # (the end token itself is never appended)
            assert int(s.lens[b]) == len(held)
    # every beam's pages hold its own tokens' keys and values, in both layers
    for b in range(s.n):
        held = beams[b] if not ended[b] else beams[b][:-1]
        x = s.tokens_qkv[held].double().numpy().reshape(len(held), nq + 2 * nkv, hd)
        for layer in range(2):
            k, v = s.rows(b, layer)
            want = torch.from_numpy(x[:, nq + nkv:] * (1 + layer)).to(ref.torch_dtype(io)).to(ref.torch_dtype(cache)).double().numpy()
            np.testing.assert_array_equal(v, want)
            y = ref.rope(x[:, nq:nq + nkv] * (1 + layer), np.arange(len(held)), s.freqs, False, s.mscale, hd)
            half = ref.EPS_HALF[cache] * 2 + 8 * ref.U
            np.testing.assert_allclose(k, y, rtol=0, atol=half * np.abs(y).max() + ref.TINY[cache])


@pytest.mark.parametrize("io,cache,nq,nkv,hd,page", [("bf16", "bf16", 14, 2, 128, 16), ("f32", "f16", 4, 2, 64, 5)])
def test_two_steps_as_a_graph(io, cache, nq, nkv, hd, page):
    """Twelve steps, called one by one and as replays of two captured ones: the same bits, whatever the beams do."""
    G, W, vocab, prompts = 2, 5, 97, [70, 41]

    def begin():
        s = Search(G, W, nq, nkv, hd, page, 200, 40, vocab, io, cache, 40)
        s.new.zero_()
        s.new[::W] = torch.tensor(prompts, dtype=torch.int32, device="cuda")
        s.append(torch.from_numpy(np.random.default_rng(1).integers(0, vocab, sum(prompts))).cuda(), sum(prompts))
        s.shared.copy_(torch.tensor(np.repeat(prompts, W), dtype=torch.int32))
        first_q = s.q[torch.cumsum(torch.tensor(prompts), 0).cuda() - 1].clone()
        s.q[:s.n].zero_()
        s.q[0:s.n:W] = first_q
        s.scores[::W] = 0.0
        s.new.fill_(1)
        return s

    def step(s):
        s.attend()
        s.select(-1)
        s.fork()
        s.append(s.tokens, s.n)

    a, b = begin(), begin()
    for _ in range(12):
        step(a)
    step(b)
    step(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
        step(b)
    for _ in range(5):
        g.replay()
    a.check_pool()
    b.check_pool()
    assert a.hlens.tolist() == b.hlens.tolist() == [12] * a.n
    for name in ("history", "scores", "lens", "n_free", "shares", "parents"):
        x, y = getattr(a, name), getattr(b, name)
        if name == "history":
            x, y = x[:, :12], y[:, :12]
        assert torch.equal(x, y), name
    assert torch.equal(a.free[:int(a.n_free)], b.free[:int(b.n_free)])
    for w in range(a.n):
        for layer in range(2):
            for x, y in zip(a.rows(w, layer), b.rows(w, layer)):
                np.testing.assert_array_equal(x, y)
