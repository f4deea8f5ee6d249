"""The serving operators around a paged key-value cache, as they are measured: page plans, rotary
positions with the append into the cache, attention of one new token over the pages, and log
probabilities of tokens.

`run` computes each operator in plain torch (32 bits, rounded once) where `own` is false, and through
the framework's calls where it is true. `exact` computes the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"f32": 0, "bf16": 1, "f16": 2}  # the framework's type numbers
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
TURN = 2.0 * math.pi

# ---- the cases ---------------------------------------------------------------------------------------


def listed():
    attn = dict(op="attention", layout="head", idle=False)
    plan = dict(op="plan", idle=True)
    rope = dict(op="rope", factor=1.0, orig=4096)
    return [
        # one sequence just past its prompt, the model's own activations (fp32) and cache (fp16): latency
        dict(attn, name="attn_1x178", n=1, lo=178, hi=178, nq=12, nkv=2, hd=128, page=16, cache="f16", io="f32"),
        # the batched workload's ragged lengths, one layer
        dict(attn, name="attn_16x256-2048", n=16, lo=256, hi=2048, nq=12, nkv=2, hd=128, page=16, cache="f16", io="f32"),
        # a serving batch near a memory limit: 256 sequences of up to 8192 positions
        dict(attn, name="attn_256x8192_bf16", n=256, lo=1, hi=8192, nq=28, nkv=4, hd=128, page=64, cache="bf16", io="bf16"),
        # one very long context, pages as the positions lie ([page][position][head])
        dict(attn, name="attn_1x131071", n=1, lo=131071, hi=131071, nq=12, nkv=2, hd=128, page=128, cache="f16", io="f16", layout="position"),
        # an fp32 model's cache with small heads, odd pages and idle sequences
        dict(attn, name="attn_200_f32", n=200, lo=1, hi=1500, nq=6, nkv=2, hd=32, page=7, cache="f32", io="f32", idle=True),
        # a decode step of many sequences: one token each
        dict(plan, name="plan_decode_512", n=512, lo=1, hi=8000, new_lo=1, new_hi=1, page=16, blocks=512, tokens=512),
        # a prefill step: ragged prompts, some sequences idle, the token buffers larger than the prompts
        dict(plan, name="plan_prefill_64", n=64, lo=0, hi=600, new_lo=1, new_hi=4000, page=16, blocks=512, tokens=160000),
        # finished sequences give their pages back
        dict(op="release", name="release_512", n=512, lo=0, hi=8000, page=16, blocks=512, idle=True),
        # the new tokens of a batch: fp32 projections into the fp16 cache
        dict(rope, name="rope_16", tokens=16, pad=0, far=4000, nq=12, nkv=2, hd=128, rot=128, pairs="half", scaling="none", page=16, cache="f16", io="f32"),
        # a long prefill far into a scaled context, half of each head rotated in adjacent pairs
        dict(rope, name="rope_8191_bf16", tokens=8191, pad=55, far=100000, nq=28, nkv=4, hd=128, rot=64, pairs="adjacent", scaling="yarn", factor=8.0, orig=16384,
             page=64, cache="bf16", io="bf16"),
        # the sampled token of one sequence, with five alternatives
        dict(op="logprobs", name="logprobs_1", rows=1, vocab=151936, ids=1, top=5, io="f32", masked=False),
        # the tokens of a prompt scored, two candidates a position, twenty alternatives, some tokens banned
        dict(op="logprobs", name="logprobs_1024_bf16", rows=1024, vocab=152064, ids=2, top=20, io="bf16", masked=True),
    ]


HEADS = [(12, 2), (14, 2), (28, 4), (8, 2), (4, 4), (3, 1), (16, 1), (9, 3)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "plan", "release", "rope", "rope", "logprobs", "logprobs"])
    if op == "attention":
        nq, nkv = rng.choice(HEADS)
        cache, io = rng.choice([("f16", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        hd = rng.choice([64, 128, 128, 32, 96, 80, 16])
        page = rng.choice([16, 32, 64, 128, 1, 5, 24, 256])
        n = _log(rng, 1, 256)
        room = min(2 ** 30, 2 ** 30 * 2 // SIZE[cache]) // (n * nkv * hd)  # positions a sequence may have
        hi = _log(rng, 1, max(2, min(131072, room)))
        lo = rng.choice([1, hi, max(1, hi // 4)])
        return dict(op=op, n=n, lo=lo, hi=hi, nq=nq, nkv=nkv, hd=hd, page=page, cache=cache, io=io,
                    layout=rng.choice(["head", "position"]), idle=n > 4 and rng.random() < 0.3)
    if op in ("plan", "release"):
        n, page = _log(rng, 1, 2048), rng.choice([16, 32, 64, 128, 1, 7])
        hi = _log(rng, 1, min(8192, 2 ** 20 // n * page, 512 * page))
        if op == "release":
            return dict(op=op, n=n, lo=0, hi=hi, page=page, blocks=-(-hi // page) + rng.randrange(3), idle=True)
        new = rng.choice([1, _log(rng, 1, max(1, 160000 // n))])
        return dict(op=op, n=n, lo=0, hi=hi, new_lo=rng.choice([1, new]), new_hi=new, page=page, blocks=-(-(hi + new) // page) + rng.randrange(3),
                    idle=rng.random() < 0.5, tokens=n * new + rng.randrange(50))
    if op == "rope":
        nq, nkv = rng.choice(HEADS)
        cache, io = rng.choice([("f16", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        hd = rng.choice([64, 128, 128, 96, 32])
        tokens = _log(rng, 1, max(2, min(8192, 8192 * 32 * 128 * 2 // ((nq + nkv) * hd * SIZE[io]))))
        return dict(op=op, tokens=tokens, pad=rng.choice([0, tokens // 10]), far=_log(rng, 1, 1000000), nq=nq, nkv=nkv, hd=hd, rot=rng.choice([hd, hd // 2, hd // 4 * 3]),
                    pairs=rng.choice(["half", "adjacent"]), scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]), factor=rng.choice([2.0, 4.0, 32.0]),
                    orig=rng.choice([4096, 8192, 32768]), page=rng.choice([16, 64, 1, 7]), cache=cache, io=io)
    io = rng.choice(["f32", "f32", "bf16", "f16"])
    vocab = rng.choice([151936, 152064, 32000, _log(rng, 250, 152064)])
    rows = _log(rng, 1, min(4096, 1024 * 152064 * 2 // (vocab * SIZE[io])))
    return dict(op=op, rows=rows, vocab=vocab, ids=rng.choice([1, 1, 2, 5]), top=min(vocab, rng.choice([0, 1, 5, 20, 32])), io=io, masked=rng.random() < 0.5)


def _lengths(case, what="lens"):
    """The case's lengths: the same for every seed, so that the work is the case's."""
    lo, hi = (case["lo"], case["hi"]) if what == "lens" else (case["new_lo"], case["new_hi"])
    v = np.random.default_rng([case["n"], lo, hi, len(what)]).integers(lo, hi + 1, case["n"])
    if case["idle"]:
        v[(3 if what == "lens" else 5)::8] = 0
    return v.astype(np.int64)


# ---- what a program has in hand ----------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": dict(case), "err": torch.zeros(1, dtype=torch.int32, device=DEV)}
    return {"attention": _prepare_attention, "plan": _prepare_plan, "release": _prepare_plan, "rope": _prepare_rope, "logprobs": _prepare_logprobs}[case["op"]](case, gen, rng, s)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _pages(case, n_pages, gen, empty=False):
    """Keys and values of a cache of n_pages pages, `empty` of zeros."""
    shape = (n_pages, case["nkv"], case["page"], case["hd"]) if case.get("layout", "head") == "head" else (n_pages, case["page"], case["nkv"], case["hd"])
    if empty:
        return [torch.zeros(shape, dtype=TORCH[case["cache"]], device=DEV) for _ in range(2)]
    return [torch.randn(shape, dtype=TORCH[case["cache"]], device=DEV, generator=gen) for _ in range(2)]


def _paged_kv(case, kc, vc):
    from qwen2_decoder_forward_decode_gb300 import binding
    st = kc.stride()
    head, pos = (st[1], st[2]) if case.get("layout", "head") == "head" else (st[2], st[1])
    return binding.PagedKV(kc.data_ptr(), vc.data_ptr(), CODE[case["cache"]], kc.shape[0], case["page"], case["nkv"], case["hd"], st[0], head, pos)


def _prepare_attention(case, gen, rng, s):
    lens = rng.permutation(_lengths(case))
    n, page = case["n"], case["page"]
    need = -(-lens // page)
    n_pages, blocks = int(need.sum()) + 3, int(need.max())
    order = rng.permutation(n_pages)
    table = np.full((n, max(1, blocks)), 0, dtype=np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(n):
        table[b, :need[b]] = order[at[b]:at[b + 1]]
    s["kc"], s["vc"] = _pages(case, n_pages, gen)
    # queries sharp enough that a few positions carry the weight, as trained heads have them
    q = 1.5 * torch.randn(n, case["nq"], case["hd"], device=DEV, generator=gen)
    s["q"] = q.to(TORCH[case["io"]])
    s["table"], s["lens"] = _i32(table), _i32(lens)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(n, case["nq"], device=DEV)
    if own:
        from qwen2_decoder_forward_decode_gb300 import binding
        s["kv"] = _paged_kv(case, s["kc"], s["vc"])
        s["ws"] = torch.zeros(binding.paged_attention_workspace(case["nq"], case["nkv"], case["hd"]), dtype=torch.uint8, device=DEV)
    return s


def _prepare_plan(case, gen, rng, s):
    lens = _lengths(case)
    n, page, blocks = case["n"], case["page"], case["blocks"]
    turn = int(rng.integers(0, n))
    lens = np.roll(lens, turn)
    have = -(-lens // page)
    new = np.roll(_lengths(case, "new"), turn) if case["op"] == "plan" else np.zeros(n, dtype=np.int64)
    want = -(-(lens + new) // page) - have
    n_pages = int(have.sum() + want.sum()) + 17
    order = rng.permutation(n_pages).astype(np.int32)
    at = np.concatenate([[0], np.cumsum(have)])
    table = np.full((n, blocks), -1, dtype=np.int32)
    for b in range(n):
        table[b, :have[b]] = order[at[b]:at[b + 1]]
    n_free = n_pages - int(have.sum())
    free = np.full(n_pages, -1, dtype=np.int32)
    free[:n_free] = order[at[n]:]
    s["n_pages"] = n_pages
    s["lens"], s["free"], s["n_free"], s["table"] = _i32(lens), _i32(free), _i32([n_free]), _i32(table)
    s["lens_out"], s["n_free_out"] = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    if case["op"] == "release":
        s["done"] = _i32(rng.integers(0, 3, n) == 0)
    else:
        s["new"] = _i32(new)
        s["cu"] = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
        s["positions"] = torch.zeros(case["tokens"], dtype=torch.int32, device=DEV)
        s["slots"] = torch.zeros(case["tokens"], dtype=torch.int64, device=DEV)
    return s


def _prepare_rope(case, gen, rng, s):
    n, nq, nkv, hd, page = case["tokens"], case["nq"], case["nkv"], case["hd"], case["page"]
    n_pages = -(-n // page) + 2
    s["kc"], s["vc"] = _pages(case, n_pages, gen, empty=True)
    # one fused projection's output: q, k and v of a token lie in one row
    s["qkv"] = torch.randn(n, (nq + 2 * nkv) * hd, device=DEV, generator=gen).to(TORCH[case["io"]])
    s["q_out"] = torch.empty(n, nq, hd, dtype=TORCH[case["io"]], device=DEV)
    first = case["far"] + int(rng.integers(0, 1000))
    s["positions"] = _i32(first + np.arange(n))
    order = rng.permutation(n_pages)
    t = np.arange(n, dtype=np.int64)
    slots = order[t // page] * page + t % page
    slots[n - case["pad"]:] = -1
    s["slots"] = torch.from_numpy(slots).to(DEV)
    s["freqs"] = torch.from_numpy(_inverse_frequencies(case)).to(DEV)
    s["mscale"] = 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0
    if own:
        from qwen2_decoder_forward_decode_gb300 import binding
        s["kv"] = _paged_kv(case, s["kc"], s["vc"])
        turns, s["mscale"] = binding.rope_turns(case["rot"], 1e6, case["scaling"], factor=case["factor"], orig_len=case["orig"])
        s["turns"] = torch.from_numpy(turns.view(np.int64)).to(DEV)
    return s


def _prepare_logprobs(case, gen, rng, s):
    rows, vocab = case["rows"], case["vocab"]
    # a wide bulk with a few likely tokens above it
    z = 2.0 * torch.randn(rows, vocab, device=DEV, generator=gen)
    hot = torch.randint(0, vocab, (rows, min(8, vocab)), device=DEV, generator=gen)
    z.scatter_add_(1, hot, 6.0 + 2.0 * torch.rand(hot.shape, device=DEV, generator=gen))
    ids = torch.randint(0, vocab, (rows, case["ids"]), device=DEV, generator=gen)
    ids[:, 0] = hot[:, 0]
    if case["masked"]:
        ban = torch.rand(vocab, device=DEV, generator=gen) < 0.02
        ban[ids.reshape(-1)] = False
        z[:, ban] = -math.inf
    s["logits"] = z.to(TORCH[case["io"]])
    s["ids"] = ids.to(torch.int32)
    k = case["top"]
    s["logprobs"] = torch.empty(rows, case["ids"], device=DEV)
    s["ranks"] = torch.empty(rows, case["ids"], dtype=torch.int32, device=DEV)
    s["entropy"] = torch.empty(rows, device=DEV)
    s["top_ids"] = torch.empty(rows, k, dtype=torch.int32, device=DEV)
    s["top_logprobs"] = torch.empty(rows, k, device=DEV)
    if own:
        from qwen2_decoder_forward_decode_gb300 import binding
        s["ws"] = torch.zeros(binding.token_logprobs_workspace(rows, vocab, k), dtype=torch.uint8, device=DEV)
    return s


# ---- one pass ----------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "plan": _own_plan, "release": _own_release, "rope": _own_rope, "logprobs": _own_logprobs}[op](state)
    return {"attention": _plain_attention, "plan": _plain_plan, "release": _plain_release, "rope": _plain_rope, "logprobs": _plain_logprobs}[op](state)


def _own_attention(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    c = s["case"]
    binding.paged_attention(s["kv"], c["n"], c["nq"], s["table"].data_ptr(), s["table"].shape[1], s["lens"].data_ptr(), CODE[c["io"]], s["q"].data_ptr(), c["nq"] * c["hd"],
                            1.0 / math.sqrt(c["hd"]), s["out"].data_ptr(), c["nq"] * c["hd"], s["lse"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(), s["err"].data_ptr(),
                            torch.cuda.current_stream().cuda_stream)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_attention(s):
    c = s["case"]
    nkv, group, hd, page = c["nkv"], c["nq"] // c["nkv"], c["hd"], c["page"]
    kc, vc = (s["kc"].transpose(1, 2), s["vc"].transpose(1, 2)) if c["layout"] == "head" else (s["kc"], s["vc"])
    at = torch.arange(s["table"].shape[1] * page, device=DEV)
    pages, offs = s["table"].long()[:, at // page], at % page
    open_ = at[None, :] < s["lens"].long()[:, None]  # [n, L]
    k = kc[pages, offs].float()  # [n, L, nkv, hd]
    v = vc[pages, offs].float().masked_fill(~open_[:, :, None, None], 0.0)
    q = s["q"].float().view(c["n"], nkv, group, hd)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(hd))  # [n, nkv, group, L]
    z = z.masked_fill(~open_[:, None, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m.clamp_min(torch.finfo(torch.float32).min))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total.clamp_min(torch.finfo(torch.float32).tiny)
    lse = (m + torch.log(total)).view(c["n"], c["nq"])
    return {"out": o.reshape(c["n"], c["nq"], hd).to(s["q"].dtype), "lse": lse}


def _own_plan(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    c = s["case"]
    binding.page_plan(c["n"], c["page"], s["n_pages"], c["blocks"], c["tokens"], s["lens"].data_ptr(), s["new"].data_ptr(), s["free"].data_ptr(), s["n_free"].data_ptr(),
                      s["table"].data_ptr(), s["lens_out"].data_ptr(), s["n_free_out"].data_ptr(), s["cu"].data_ptr(), s["positions"].data_ptr(), s["slots"].data_ptr(),
                      s["err"].data_ptr(), torch.cuda.current_stream().cuda_stream)
    return {"table": s["table"], "lens": s["lens_out"], "n_free": s["n_free_out"], "cu": s["cu"], "positions": s["positions"], "slots": s["slots"]}


def _plain_plan(s):
    c = s["case"]
    page, n = c["page"], c["n"]
    lens, new = s["lens"].long(), s["new"].long()
    have, need = (lens + page - 1) // page, (lens + new + page - 1) // page
    before = torch.cumsum(need - have, 0) - (need - have)  # pages taken by the sequences before
    col = torch.arange(c["blocks"], device=DEV)
    fresh = (col >= have[:, None]) & (col < need[:, None])
    pick = s["n_free"].long() - 1 - (before[:, None] + col - have[:, None])
    table = torch.where(fresh, s["free"][pick.clamp(0, s["n_pages"] - 1)], s["table"])
    ends = torch.cumsum(new, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), ends])
    t = torch.arange(c["tokens"], device=DEV)
    b = torch.searchsorted(ends, t, right=True).clamp_max(n - 1)
    real = t < ends[-1]
    pos = torch.where(real, lens[b] + t - cu[b], 0)
    slots = torch.where(real, table[b, (pos // page).clamp_max(c["blocks"] - 1)].long() * page + pos % page, -1)
    return {"table": table, "lens": (lens + new).to(torch.int32), "n_free": s["n_free"] - (need - have).sum().to(torch.int32), "cu": cu.to(torch.int32),
            "positions": pos.to(torch.int32), "slots": slots}


def _own_release(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    c = s["case"]
    binding.page_release(c["n"], c["page"], s["n_pages"], c["blocks"], s["lens"].data_ptr(), s["done"].data_ptr(), s["table"].data_ptr(), s["free"].data_ptr(), s["n_free"].data_ptr(),
                         s["lens_out"].data_ptr(), s["n_free_out"].data_ptr(), s["err"].data_ptr(), torch.cuda.current_stream().cuda_stream)
    return {"free": s["free"], "lens": s["lens_out"], "n_free": s["n_free_out"]}


def _plain_release(s):
    c = s["case"]
    page = c["page"]
    lens, done = s["lens"].long(), s["done"].bool()
    gone = torch.where(done, (lens + page - 1) // page, 0)
    before = torch.cumsum(gone, 0) - gone
    col = torch.arange(c["blocks"], device=DEV)
    mine = col < gone[:, None]
    to = torch.where(mine, s["n_free"].long() + before[:, None] + col, s["n_pages"])  # the last place is thrown away
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free[to.reshape(-1)] = s["table"].reshape(-1)
    return {"free": free[:-1], "lens": torch.where(done, 0, lens).to(torch.int32), "n_free": s["n_free"] + gone.sum().to(torch.int32)}


def _own_rope(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    c = s["case"]
    nq, nkv, hd, size = c["nq"], c["nkv"], c["hd"], SIZE[c["io"]]
    q, row = s["qkv"].data_ptr(), (nq + 2 * nkv) * hd
    binding.rope_append(s["kv"], c["tokens"], nq, CODE[c["io"]], s["positions"].data_ptr(), s["slots"].data_ptr(), s["turns"].data_ptr(), c["rot"], c["pairs"] == "adjacent", s["mscale"],
                        q, row, q + nq * hd * size, row, q + (nq + nkv) * hd * size, row, s["q_out"].data_ptr(), nq * hd, s["err"].data_ptr(),
                        torch.cuda.current_stream().cuda_stream)
    return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}


def _inverse_frequencies(c):
    """theta^(-2i/r) and its scaled forms, in 64 bits."""
    r, theta, f, orig = c["rot"], 1e6, c["factor"], c["orig"]
    i = np.arange(r // 2, dtype=np.float64)
    if c["scaling"] == "ntk":
        theta = theta * f ** (r / (r - 2)) if r > 2 else theta
    inv = theta ** (-2 * i / r)
    if c["scaling"] == "linear":
        inv = inv / f
    elif c["scaling"] == "yarn":  # between beta_fast = 32 and beta_slow = 1 turns over the original length
        lo, hi = (r * math.log(orig / (beta * TURN)) / (2 * math.log(theta)) for beta in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), r - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        inv = inv / f * ramp + inv * (1 - ramp)
    elif c["scaling"] == "bands":  # wavelengths over orig are divided, those under orig / 4 kept
        turns = orig * inv / TURN
        mix = np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1)
        inv = (1 - mix) * inv / f + mix * inv
    return inv


def _plain_rope(s):
    c = s["case"]
    n, nq, nkv, hd, r, page = c["tokens"], c["nq"], c["nkv"], c["hd"], c["rot"], c["page"]
    x = s["qkv"].float().view(n, nq + 2 * nkv, hd)
    angle = s["positions"].double()[:, None] * s["freqs"]  # 64 bits: far positions
    cos, sin = (torch.cos(angle) * s["mscale"]).float()[:, None], (torch.sin(angle) * s["mscale"]).float()[:, None]
    a, b = (x[:, :nq + nkv, 0:r:2], x[:, :nq + nkv, 1:r:2]) if c["pairs"] == "adjacent" else (x[:, :nq + nkv, :r // 2], x[:, :nq + nkv, r // 2:r])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([ra, rb], -1).flatten(-2) if c["pairs"] == "adjacent" else torch.cat([ra, rb], -1)
    y = torch.cat([y, x[:, :nq + nkv, r:]], -1)
    n_pages = s["kc"].shape[0]
    at = torch.where(s["slots"] >= 0, s["slots"], n_pages * page)  # the last place is thrown away

    def put(cache, rows):  # [n_pages, nkv, page, hd] as rows of positions
        flat = torch.cat([cache.transpose(1, 2).reshape(n_pages * page, nkv, hd), cache.new_zeros(1, nkv, hd)])
        flat[at] = rows.to(cache.dtype)
        return flat[:-1].view(n_pages, page, nkv, hd).transpose(1, 2).contiguous()

    return {"q": y[:, :nq].to(s["qkv"].dtype), "k": put(s["kc"], y[:, nq:]), "v": put(s["vc"], x[:, nq + nkv:])}


def _own_logprobs(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    c = s["case"]
    binding.token_logprobs(CODE[c["io"]], c["rows"], c["vocab"], s["logits"].data_ptr(), c["vocab"], s["ids"].data_ptr(), c["ids"], s["logprobs"].data_ptr(), s["ranks"].data_ptr(),
                           s["entropy"].data_ptr(), c["top"], s["top_ids"].data_ptr(), s["top_logprobs"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(), s["err"].data_ptr(),
                           torch.cuda.current_stream().cuda_stream)
    return {"logprobs": s["logprobs"], "ranks": s["ranks"], "entropy": s["entropy"], "top_ids": s["top_ids"], "top_logprobs": s["top_logprobs"]}


def _plain_logprobs(s):
    c = s["case"]
    z = s["logits"].float() + 0.0  # -0 and 0 are one value
    ids = s["ids"].long()
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    logz = torch.log(total)
    given = z.gather(1, ids)
    ent = logz[:, 0] - (torch.where(e > 0, e * (z - m), 0.0)).sum(-1) / total[:, 0]
    col = torch.arange(c["vocab"], device=DEV)
    above = (z[:, None, :] > given[:, :, None]) | ((z[:, None, :] == given[:, :, None]) & (col < ids[:, :, None]))
    bits = z.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32 + (2 ** 31 - col)  # larger value, then lower index
    top = torch.topk(order, c["top"], dim=-1).values
    top_ids = 2 ** 31 - top % 2 ** 32
    return {"logprobs": given - m - logz, "ranks": (1 + above.sum(-1)).to(torch.int32), "entropy": ent, "top_ids": top_ids.to(torch.int32),
            "top_logprobs": z.gather(1, top_ids) - m - logz}


# ---- the definitions in 64 bits ----------------------------------------------------------------------


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"attention": _exact_attention, "plan": _exact_plan, "release": _exact_release, "rope": _exact_rope, "logprobs": _exact_logprobs}[case["op"]](case, s)


def _exact_attention(c, s):
    group, page = c["nq"] // c["nkv"], c["page"]
    out = torch.zeros(c["n"], c["nq"], c["hd"], dtype=torch.float64, device=DEV)
    lse = torch.full((c["n"], c["nq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b, length in enumerate(s["lens"].tolist()):
        if not length:
            continue
        rows = s["table"][b, :-(-length // page)].long()
        for g in range(c["nkv"]):
            k, v = ((x[rows, g] if c["layout"] == "head" else x[rows, :, g]).reshape(-1, c["hd"])[:length].double() for x in (s["kc"], s["vc"]))
            heads = slice(g * group, (g + 1) * group)
            z = s["q"][b, heads].double() @ k.T / math.sqrt(c["hd"])
            lse[b, heads] = torch.logsumexp(z, -1)
            out[b, heads] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse}


def _exact_plan(c, s):
    lens, new, table, page = s["lens"].tolist(), s["new"].tolist(), s["table"].cpu().numpy().copy(), c["page"]
    free = s["free"].tolist()[:int(s["n_free"])]
    cu, slots, positions = [0], [], []
    for b in range(c["n"]):
        for j in range(-(-lens[b] // page), -(-(lens[b] + new[b]) // page)):
            table[b, j] = free.pop()
        at = np.arange(lens[b], lens[b] + new[b])
        positions.append(at)
        slots.append(table[b, at // page].astype(np.int64) * page + at % page)
        cu.append(cu[-1] + new[b])
    rest = c["tokens"] - cu[-1]
    return {"table": table, "lens": np.array(lens, dtype=np.int32) + np.array(new, dtype=np.int32), "n_free": np.array([len(free)], dtype=np.int32), "cu": np.array(cu, dtype=np.int32),
            "positions": np.concatenate(positions + [np.zeros(rest)]).astype(np.int32), "slots": np.concatenate(slots + [np.full(rest, -1)]).astype(np.int64)}


def _exact_release(c, s):
    lens, done, table = s["lens"].tolist(), s["done"].tolist(), s["table"].cpu().numpy()
    free, at = s["free"].cpu().numpy().copy(), int(s["n_free"])
    for b in range(c["n"]):
        pages = -(-lens[b] // c["page"]) if done[b] else 0
        free[at:at + pages] = table[b, :pages]
        at += pages
    return {"free": free, "lens": np.array([0 if d else v for v, d in zip(lens, done)], dtype=np.int32), "n_free": np.array([at], dtype=np.int32)}


def _exact_rope(c, s):
    n, nq, nkv, hd, r, page = c["tokens"], c["nq"], c["nkv"], c["hd"], c["rot"], c["page"]
    x = s["qkv"].double().view(n, nq + 2 * nkv, hd).cpu().numpy().copy()
    pos = s["positions"].cpu().numpy().astype(np.float64)
    scale = 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0
    for i in range(r // 2):
        w = 1e6 ** (-2.0 * i / r)
        if c["scaling"] == "linear":
            w /= c["factor"]
        elif c["scaling"] == "ntk" and r > 2:
            w *= c["factor"] ** (-2.0 * i / (r - 2))
        elif c["scaling"] == "yarn":
            edge = [r / 2 * math.log(c["orig"] / TURN / turns) / math.log(1e6) for turns in (32, 1)]
            first, last = max(0, math.floor(edge[0])), min(r - 1, math.ceil(edge[1]))
            part = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            w = w * (1 - part) + w / c["factor"] * part
        elif c["scaling"] == "bands":
            wave = TURN / w
            if wave > c["orig"]:
                w /= c["factor"]
            elif wave > c["orig"] / 4.0:
                part = (c["orig"] / wave - 1.0) / 3.0
                w = (1 - part) * w / c["factor"] + part * w
        e, f = (2 * i, 2 * i + 1) if c["pairs"] == "adjacent" else (i, i + r // 2)
        z = (x[:, :nq + nkv, e] + 1j * x[:, :nq + nkv, f]) * (scale * np.exp(1j * np.fmod(pos * w, TURN)))[:, None]
        x[:, :nq + nkv, e], x[:, :nq + nkv, f] = z.real, z.imag
    caches = []
    for cache, rows in ((s["kc"], x[:, nq:nq + nkv]), (s["vc"], x[:, nq + nkv:])):
        y = cache.double().cpu().numpy()
        slot = s["slots"].cpu().numpy()
        kept = slot[slot >= 0]
        y[kept // page, :, kept % page] = rows[slot >= 0]
        caches.append(y)
    return {"q": x[:, :nq].copy(), "k": caches[0], "v": caches[1]}


def _exact_logprobs(c, s):
    z = s["logits"].double()
    p = torch.log_softmax(z, -1)
    ids = s["ids"].long()
    entropy = -torch.where(torch.isinf(p), 0.0, torch.exp(p) * p).sum(-1)
    value, index = torch.sort(z, dim=-1, descending=True, stable=True)
    place = torch.empty_like(index).scatter_(1, index, torch.arange(1, c["vocab"] + 1, device=DEV).expand_as(index))
    return {"logprobs": p.gather(1, ids), "ranks": place.gather(1, ids).to(torch.int32), "entropy": entropy, "top_ids": index[:, :c["top"]].to(torch.int32),
            "top_logprobs": p.gather(1, index[:, :c["top"]])}


# ---- what a pass cannot do without -------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "attention":
        total = int(_lengths(c).sum())
        kv = 2 * total * c["nkv"] * c["hd"] * SIZE[c["cache"]]
        ends = 2 * c["n"] * c["nq"] * c["hd"] * SIZE[c["io"]] + 4 * c["n"] * (c["nq"] + 1)
        return {"bytes": kv + ends + 4 * (total // c["page"]), "flops": 4 * c["nq"] * c["hd"] * total}
    if c["op"] in ("plan", "release"):
        lens = _lengths(c)
        if c["op"] == "release":  # about a third of the pages move from the tables to the list
            return {"bytes": 12 * c["n"] + 8 * int((-(-lens // c["page"])).sum()) // 3, "flops": 0}
        fresh = int((-(-(lens + _lengths(c, "new")) // c["page"]) - -(-lens // c["page"])).sum())
        return {"bytes": 16 * c["n"] + 8 * fresh + 12 * c["tokens"], "flops": 0}
    if c["op"] == "rope":
        rows = 2 * c["nq"] * SIZE[c["io"]] + 2 * c["nkv"] * (SIZE[c["io"]] + SIZE[c["cache"]])
        return {"bytes": c["tokens"] * (rows * c["hd"] + 12), "flops": 3 * c["tokens"] * (c["nq"] + c["nkv"]) * c["rot"]}
    read = c["rows"] * c["vocab"] * SIZE[c["io"]]
    return {"bytes": read + c["rows"] * (12 * c["ids"] + 8 * c["top"] + 4), "flops": 5 * c["rows"] * c["vocab"]}
