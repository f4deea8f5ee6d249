"""The operators that let several continuations of one prompt live in a paged cache, as they are measured:
attention of groups that share a prompt, beam selection, forks of sequences with counted pages, copies of
pages, and compaction of the pool.

`run` computes each operator in plain torch (32 bits, 64 where an order depends on them) where `own` is
false, and through the framework's calls where it is true. `exact` computes the same from the definitions
in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"f32": 0, "bf16": 1, "f16": 2}  # the framework's type numbers
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
END = 7  # the token that ends a beam

# ---- the cases ---------------------------------------------------------------------------------------


def listed():
    shared = dict(op="shared", layout="head", idle=False)
    beam = dict(op="beam", masked=False)
    return [
        # four beams of one request just past its prompt, the model's own activations (fp32) and cache (fp16): latency
        dict(shared, name="shared_1x4", groups=1, each_lo=4, each_hi=4, pre_lo=178, pre_hi=178, own_lo=1, own_hi=24, nq=12, nkv=2, hd=128, page=16, cache="f16", io="f32"),
        # a serving batch: 16 prompts with eight samples each
        dict(shared, name="shared_16x8_bf16", groups=16, each_lo=8, each_hi=8, pre_lo=512, pre_hi=4096, own_lo=1, own_hi=512, nq=28, nkv=4, hd=128, page=64, cache="bf16", io="bf16"),
        # one long system prompt before 256 users' short turns
        dict(shared, name="shared_1x256_bf16", groups=1, each_lo=256, each_hi=256, pre_lo=16383, pre_hi=16383, own_lo=1, own_hi=256, nq=28, nkv=4, hd=128, page=64, cache="bf16", io="bf16"),
        # an fp32 model's cache, odd heads and pages, ragged groups, idle sequences, pages as the positions lie
        dict(shared, name="shared_5_f32", groups=5, each_lo=1, each_hi=30, pre_lo=1, pre_hi=1500, own_lo=0, own_hi=300, nq=9, nkv=3, hd=80, page=7, cache="f32", io="f32",
             layout="position", idle=True),
        # one request of four beams, twice as many candidates as beams, the model's fp32 logits: latency
        dict(beam, name="beam_1x4", groups=1, beams=4, vocab=151936, n_out=8, io="f32", width=256, first=False, weights=False, end=True),
        # 64 requests of four beams, ended beams weighed by their length, some tokens banned
        dict(beam, name="beam_64x4_bf16", groups=64, beams=4, vocab=152064, n_out=4, io="bf16", width=512, first=False, weights=True, end=True, masked=True),
        # a prompt becomes sixteen samples
        dict(op="fork", name="fork_1x16", groups=1, beams=1, n_out=16, pre_lo=1001, pre_hi=1001, own_lo=0, own_hi=0, page=16, blocks=128, idle=False),
        # a step of beam search: 64 requests of four beams take their parents' pages, some requests are done
        dict(op="fork", name="fork_64x4", groups=64, beams=4, n_out=4, pre_lo=100, pre_hi=6000, own_lo=1, own_hi=2000, page=16, blocks=512, idle=True),
        # the last pages of sixteen new samples, partly filled, in all layers of the small model
        dict(op="copy", name="copy_16x28", n=16, pages=48, layers=28, nkv=2, hd=128, page=16, cache="f16", layout="head", filled=True),
        # whole pages moved by a compaction
        dict(op="copy", name="copy_256x12_bf16", n=256, pages=520, layers=12, nkv=4, hd=128, page=64, cache="bf16", layout="position", filled=False),
        # a small pool, all holes closed
        dict(op="compact", name="compact_4096", pages=4096, n=64, live=0.6, page=16, blocks=64, moves=2048),
        # a million pages of 2048 sequences, a bounded number of moves
        dict(op="compact", name="compact_1m", pages=1048576, n=2048, live=0.55, page=16, blocks=512, moves=65536),
    ]


HEADS = [(12, 2), (14, 2), (28, 4), (8, 2), (4, 4), (3, 1), (16, 1), (9, 3)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "beam", "beam", "beam", "fork", "copy", "compact"])
    if op == "shared":
        nq, nkv = rng.choice(HEADS)
        cache, io = rng.choice([("f16", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        hd = rng.choice([64, 128, 128, 32, 96, 80, 16])
        groups, each = _log(rng, 1, 64), _log(rng, 1, 256)
        each = max(1, min(each, 1024 // groups))
        n, row = groups * each, nkv * hd * SIZE[cache] * 2
        flops = 2e10 if cache == "f32" else 5e10
        pre = _log(rng, 1, max(2, min(32768, int(flops / (4 * nq * hd * n)), 10 ** 8 // (row * groups))))
        own_hi = _log(rng, 1, max(2, min(2048, 5 * 10 ** 7 // (row * n))))
        return dict(op=op, groups=groups, each_lo=rng.choice([1, each]), each_hi=each, pre_lo=rng.choice([0, pre, max(1, pre // 4)]), pre_hi=pre, own_lo=rng.choice([0, 1, own_hi]),
                    own_hi=own_hi, nq=nq, nkv=nkv, hd=hd, page=rng.choice([16, 32, 64, 128, 1, 5, 24, 256]), cache=cache, io=io, layout=rng.choice(["head", "position"]),
                    idle=rng.random() < 0.3)
    if op == "beam":
        io = rng.choice(["f32", "f32", "bf16", "f16"])
        vocab = rng.choice([151936, 152064, 32000, _log(rng, 250, 152064)])
        beams = rng.choice([1, 2, 3, 4, 4, 5, 8, 16, 32])
        groups = _log(rng, 1, max(1, min(512, 256 * 152064 * 2 // (vocab * SIZE[io] * beams))))
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, n_out=rng.choice([beams, min(32, 2 * beams)]), io=io, width=_log(rng, 2, 1024), first=rng.random() < 0.2,
                    weights=rng.random() < 0.5, end=rng.random() < 0.7, masked=rng.random() < 0.4)
    if op == "fork":
        groups, beams, page = _log(rng, 1, 128), rng.choice([1, 2, 4, 5, 8]), rng.choice([16, 32, 64, 128, 1, 7])
        room = min(512 * page, 10 ** 6 // (groups * beams) * page)
        pre, tail = _log(rng, 1, room * 3 // 4), _log(rng, 1, max(1, room // 4))
        return dict(op=op, groups=groups, beams=beams, n_out=rng.choice([beams, beams, 2 * beams, 16]), pre_lo=rng.choice([0, pre]), pre_hi=pre, own_lo=0, own_hi=tail, page=page,
                    blocks=-(-(pre + tail) // page) + rng.randrange(3), idle=rng.random() < 0.5)
    if op == "copy":
        nkv, hd, page = rng.choice([1, 2, 4, 3]), rng.choice([64, 128, 96, 80, 8]), rng.choice([16, 32, 64, 1, 7])
        cache = rng.choice(["f16", "bf16", "f32"])
        layers = rng.choice([1, 12, 24, 28, 5])
        n = _log(rng, 1, min(1024, 200 * 10 ** 6 // (layers * nkv * hd * page * SIZE[cache])))
        return dict(op=op, n=n, pages=2 * n + rng.randrange(9), layers=layers, nkv=nkv, hd=hd, page=page, cache=cache, layout=rng.choice(["head", "position"]), filled=rng.random() < 0.5)
    pages = _log(rng, 64, 1048576)
    n, blocks = _log(rng, 1, min(2048, pages // 8)), 512
    return dict(op=op, pages=pages, n=n, live=rng.choice([0.1, 0.5, 0.9]), page=rng.choice([16, 32, 64, 1, 7]), blocks=blocks, moves=rng.choice([pages // 2, _log(rng, 1, pages // 2)]))


def _spread(tag, n, lo, hi):
    """n sizes between lo and hi, the same for every seed, so that the work is the case's."""
    return np.random.default_rng([tag, n, lo, hi]).integers(lo, hi + 1, n).astype(np.int64)


def _groups(c):
    """Sequences of each group, their first sequences, shared positions of each group, lengths of all."""
    size = _spread(1, c["groups"], c["each_lo"], c["each_hi"])
    cu = np.concatenate([[0], np.cumsum(size)])
    pre = _spread(2, c["groups"], c["pre_lo"], c["pre_hi"])
    lens = np.repeat(pre, size) + _spread(3, int(cu[-1]), c["own_lo"], c["own_hi"])
    if c["idle"]:
        lens[5::8] = 0
    return size, cu, pre, lens


# ---- what a program has in hand ----------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": dict(case), "err": torch.zeros(1, dtype=torch.int32, device=DEV)}
    return {"shared": _prepare_shared, "beam": _prepare_beam, "fork": _prepare_fork, "copy": _prepare_copy, "compact": _prepare_compact}[case["op"]](case, gen, rng, s)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _int(*shape):
    return torch.full(shape, -1, dtype=torch.int32, device=DEV)


def _pages(c, n_pages, gen):
    shape = (n_pages, c["nkv"], c["page"], c["hd"]) if c["layout"] == "head" else (n_pages, c["page"], c["nkv"], c["hd"])
    return [torch.randn(shape, device=DEV, generator=gen).to(TORCH[c["cache"]]) for _ in range(2)]


def _by_position(c, cache):
    """The cache as [page][position][head][dimension]."""
    return cache.transpose(1, 2) if c["layout"] == "head" else cache


def _paged_kv(c, kc, vc):
    from qwen2_decoder_forward_decode_gb300 import binding
    st = kc.stride()
    head, pos = (st[1], st[2]) if c["layout"] == "head" else (st[2], st[1])
    return binding.PagedKV(kc.data_ptr(), vc.data_ptr(), CODE[c["cache"]], kc.shape[0], c["page"], c["nkv"], c["hd"], st[0], head, pos)


def _prepare_shared(c, gen, rng, s):
    size, cu, pre, lens = _groups(c)
    n, page = len(lens), c["page"]
    need = np.maximum(-(-lens // page), np.repeat(-(-pre // page), size))  # an idle sequence's pages stay
    full = np.repeat(pre // page, size)  # pages that lie in the shared part with all their positions
    first = np.repeat(cu[:-1], size)
    fresh = np.where(np.arange(n) == first, need, need - full)
    n_pages = int(fresh.sum()) + 3
    order = rng.permutation(n_pages)
    at = np.concatenate([[0], np.cumsum(fresh)])
    table = np.zeros((n, max(1, int(need.max()))), dtype=np.int32)
    for b in range(n):
        if b == first[b]:
            table[b, :need[b]] = order[at[b]:at[b + 1]]
        else:
            table[b, :full[b]] = table[first[b], :full[b]]
            table[b, full[b]:need[b]] = order[at[b]:at[b + 1]]
    s["kc"], s["vc"] = _pages(c, n_pages, gen)
    # the page on which the shared part ends was copied for every further sequence
    rest = np.repeat(pre % page, size)
    copied = np.flatnonzero((np.arange(n) != first) & (rest > 0))
    if len(copied):
        to, src = (torch.from_numpy(table[x, full[copied]].astype(np.int64)).to(DEV) for x in (copied, first[copied]))
        keep = torch.arange(page, device=DEV)[None, :, None, None] < torch.from_numpy(rest[copied]).to(DEV)[:, None, None, None]
        for cache in (s["kc"], s["vc"]):
            rows = _by_position(c, cache)
            rows[to] = torch.where(keep, rows[src], rows[to])
    # queries sharp enough that a few positions carry the weight, as trained heads have them
    s["q"] = (1.5 * torch.randn(n, c["nq"], c["hd"], device=DEV, generator=gen)).to(TORCH[c["io"]])
    s["table"], s["lens"], s["cu"], s["shared"] = _i32(table), _i32(lens), _i32(cu), _i32(np.repeat(pre, size))
    s["cu_host"], s["pre_host"], s["own_most"] = cu.tolist(), pre.tolist(), int(max(0, (lens - np.repeat(pre, size)).max()))
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(n, c["nq"], device=DEV)
    if own:
        from qwen2_decoder_forward_decode_gb300 import binding
        s["kv"] = _paged_kv(c, s["kc"], s["vc"])
        s["ws"] = torch.zeros(binding.shared_attention_workspace(n, c["nq"], c["nkv"], c["hd"]), dtype=torch.uint8, device=DEV)
    return s


def _prepare_beam(c, gen, rng, s):
    rows, vocab, width, n_out = c["groups"] * c["beams"], c["vocab"], c["width"], c["n_out"]
    # a wide bulk with a few likely tokens above it
    z = 2.0 * torch.randn(rows, vocab, device=DEV, generator=gen)
    hot = torch.randint(0, vocab, (rows, min(8, vocab)), device=DEV, generator=gen)
    z.scatter_add_(1, hot, 6.0 + 2.0 * torch.rand(hot.shape, device=DEV, generator=gen))
    if c["end"]:
        z[::3, END] = 9.0 + torch.rand(z[::3, END].shape, device=DEV, generator=gen)
    if c["masked"]:
        ban = torch.rand(vocab, device=DEV, generator=gen) < 0.02
        ban[END] = False
        z[:, ban] = -math.inf
    s["logits"] = z.to(TORCH[c["io"]])
    first = c["first"]  # the step after the prompt: the beams are equal, and all but one are dead
    scores = -8.0 - 4.0 * torch.rand(rows, device=DEV, generator=gen)
    if first:
        scores.view(c["groups"], c["beams"])[:, 1:] = -math.inf
    s["scores"] = scores
    ended = rng.random(rows) < (0.25 if c["end"] and not first else 0.0)
    lens = rng.integers(0, width, rows)
    s["ended"], s["lens"] = _i32(ended), _i32(lens)
    s["history"] = torch.randint(0, vocab, (rows, width), device=DEV, generator=gen).to(torch.int32)
    # scores are compared over a power of the length
    s["weights"] = torch.from_numpy((1.0 / (lens + 1.0 - ended) .clip(1.0) ** 0.7).astype(np.float32)).to(DEV) if c["weights"] else None
    k = c["groups"] * n_out
    s["parents"], s["tokens"], s["ended_out"], s["lens_out"] = _int(k), _int(k), _int(k), _int(k)
    s["scores_out"], s["history_out"] = torch.empty(k, device=DEV), _int(k, width)
    if own:
        from qwen2_decoder_forward_decode_gb300 import binding
        s["ws"] = torch.zeros(binding.beam_select_workspace(c["groups"], c["beams"], vocab, n_out), dtype=torch.uint8, device=DEV)
    return s


def _prepare_fork(c, gen, rng, s):
    groups, beams, page, blocks = c["groups"], c["beams"], c["page"], c["blocks"]
    n = groups * beams
    pre = np.repeat(_spread(4, groups, c["pre_lo"], c["pre_hi"]), beams)
    lens = pre + np.repeat(_spread(5, groups, c["own_lo"], c["own_hi"]), beams)
    need, full = -(-lens // page), lens // page
    first = np.repeat(np.arange(groups) * beams, beams)
    # a beam parted from the first one somewhere behind the prompt; the pages before are one
    parted = np.where(np.arange(n) == first, 0, np.minimum(full, pre // page + rng.integers(0, np.maximum(1, full - pre // page + 1))))
    fresh = need - parted
    n_pages = int(need.sum()) + groups * c["n_out"] + 17  # the pool is the same for every seed
    order = rng.permutation(n_pages)
    at = np.concatenate([[0], np.cumsum(fresh)])
    table = np.full((n, blocks), -1, dtype=np.int32)
    for b in range(n):
        table[b, :parted[b]] = table[first[b], :parted[b]]
        table[b, parted[b]:need[b]] = order[at[b]:at[b + 1]]
    held = np.bincount(table[np.arange(blocks) < need[:, None]], minlength=n_pages)
    n_free = n_pages - int(at[-1])
    free = np.full(n_pages, -1, dtype=np.int32)
    free[:n_free] = order[at[-1]:]
    parents = np.sort(rng.integers(0, beams, (groups, c["n_out"])), axis=1) + (np.arange(groups) * beams)[:, None]
    if c["idle"]:
        parents[3::8] = -1
    s["n_pages"], s["parents"] = n_pages, _i32(parents.reshape(-1))
    s["lens"], s["table"], s["shares"], s["free"], s["n_free"] = _i32(lens), _i32(table), _i32(np.maximum(held - 1, 0)), _i32(free), _i32([n_free])
    k = groups * c["n_out"]
    s["lens_out"], s["table_out"], s["shares_out"], s["free_out"], s["n_free_out"] = _int(k), _int(k, blocks), _int(n_pages), _int(n_pages), _int(1)
    s["copy_src"], s["copy_dst"], s["copy_len"] = _int(k), _int(k), _int(k)
    if own:
        from qwen2_decoder_forward_decode_gb300 import binding
        s["ws"] = torch.zeros(binding.page_fork_workspace(n_pages), dtype=torch.uint8, device=DEV)
    return s


def _prepare_copy(c, gen, rng, s):
    s["caches"] = [_pages(c, c["pages"], gen) for _ in range(c["layers"])]
    order = rng.permutation(c["pages"])
    src, dst = order[:c["n"]].copy(), order[c["n"]:2 * c["n"]].copy()
    src[7::16] = -1  # an entry that asks for nothing
    s["src"], s["dst"] = _i32(src), _i32(dst)
    s["len"] = _i32(np.random.default_rng([6, c["n"]]).integers(1, c["page"] + 1, c["n"])) if c["filled"] else None
    if own:
        from qwen2_decoder_forward_decode_gb300 import binding
        s["kvs"] = binding.paged_kv_array([_paged_kv(c, k, v) for k, v in s["caches"]])
    return s


def _prepare_compact(c, gen, rng, s):
    n, n_pages, page, blocks = c["n"], c["pages"], c["page"], c["blocks"]
    most = min(blocks, int(2 * c["live"] * n_pages / n))
    need = _spread(7, n, 0, most)
    need = np.minimum(need, np.maximum(0, int(c["live"] * n_pages) - (np.cumsum(need) - need)))
    order = rng.permutation(n_pages)
    at = np.concatenate([[0], np.cumsum(need)])
    table = np.full((n, blocks), -1, dtype=np.int32)
    col = np.arange(blocks)
    table[col < need[:, None]] = order[:at[-1]]
    for b in range(1, n, 4):  # every fourth sequence shares its predecessor's first pages
        k = min(need[b], need[b - 1]) // 2
        table[b, :k] = table[b - 1, :k]
    mine = table[col < need[:, None]]
    held = np.bincount(mine, minlength=n_pages)
    live = int((held > 0).sum())
    free = np.full(n_pages, -1, dtype=np.int32)
    free[:n_pages - live] = rng.permutation(np.flatnonzero(held == 0))
    s["lens"] = _i32(np.maximum(0, need * page - np.minimum(page - 1, need)))
    s["table"], s["shares"], s["free"], s["n_free"] = _i32(table), _i32(np.maximum(held - 1, 0)), _i32(free), _i32([n_pages - live])
    s["table_out"], s["shares_out"], s["free_out"] = _int(n, blocks), _int(n_pages), _int(n_pages)
    s["src"], s["dst"], s["n_moves"] = _int(c["moves"]), _int(c["moves"]), _int(1)
    if own:
        from qwen2_decoder_forward_decode_gb300 import binding
        s["ws"] = torch.zeros(binding.page_compact_workspace(n_pages), dtype=torch.uint8, device=DEV)
    return s


# ---- one pass ----------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return {"shared": _own_shared, "beam": _own_beam, "fork": _own_fork, "copy": _own_copy, "compact": _own_compact}[op](state)
    return {"shared": _plain_shared, "beam": _plain_beam, "fork": _plain_fork, "copy": _plain_copy, "compact": _plain_compact}[op](state)


def _own_shared(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    c = s["case"]
    row = c["nq"] * c["hd"]
    binding.shared_attention(s["kv"], s["q"].shape[0], c["nq"], s["table"].data_ptr(), s["table"].shape[1], s["lens"].data_ptr(), c["groups"], s["cu"].data_ptr(), s["shared"].data_ptr(),
                             CODE[c["io"]], s["q"].data_ptr(), row, 1.0 / math.sqrt(c["hd"]), s["out"].data_ptr(), row, s["lse"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(),
                             s["err"].data_ptr(), torch.cuda.current_stream().cuda_stream)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_shared(s):
    """Group by group: the shared keys once for all its rows, each sequence's own behind them."""
    c = s["case"]
    nkv, grp, hd, page = c["nkv"], c["nq"] // c["nkv"], c["hd"], c["page"]
    kc, vc = _by_position(c, s["kc"]), _by_position(c, s["vc"])
    out, lse = torch.empty_like(s["q"]), torch.empty_like(s["lse"])
    scale, lowest = 1.0 / math.sqrt(hd), torch.finfo(torch.float32).min
    own_at = torch.arange(s["own_most"], device=DEV)
    for g, pre in enumerate(s["pre_host"]):
        lo, hi = s["cu_host"][g], s["cu_host"][g + 1]
        n = hi - lo
        q = s["q"][lo:hi].float().view(n, nkv, grp, hd)
        length = s["lens"][lo:hi].long()
        at = torch.arange(pre, device=DEV)
        pages = s["table"][lo].long()[at // page]
        kp, vp = kc[pages, at % page].float(), vc[pages, at % page].float()  # [pre, nkv, hd]
        pos = pre + own_at
        block = (pos // page).clamp_max(s["table"].shape[1] - 1)
        pages = s["table"][lo:hi].long()[:, block]
        open_ = pos < length[:, None]
        ko, vo = kc[pages, pos % page].float(), vc[pages, pos % page].float()  # [n, own, nkv, hd]
        vo = vo.masked_fill(~open_[:, :, None, None], 0.0)
        zp = torch.matmul(q.permute(1, 0, 2, 3).reshape(nkv, n * grp, hd), kp.permute(1, 2, 0)).view(nkv, n, grp, pre).permute(1, 0, 2, 3) * scale
        zp = zp.masked_fill((length == 0)[:, None, None, None], -math.inf)
        zo = (torch.matmul(q, ko.permute(0, 2, 3, 1)) * scale).masked_fill(~open_[:, None, None, :], -math.inf)
        z = torch.cat([zp, zo], -1)
        m = z.amax(-1, keepdim=True) if z.shape[-1] else z.new_full((n, nkv, grp, 1), -math.inf)
        p = torch.exp(z - m.clamp_min(lowest))
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p[..., :pre].permute(1, 0, 2, 3).reshape(nkv, n * grp, pre), vp.permute(1, 0, 2)).view(nkv, n, grp, hd).permute(1, 0, 2, 3)
        o = (o + torch.matmul(p[..., pre:], vo.permute(0, 2, 1, 3))) / total.clamp_min(torch.finfo(torch.float32).tiny)
        out[lo:hi] = o.reshape(n, c["nq"], hd).to(out.dtype)
        lse[lo:hi] = (m + torch.log(total)).view(n, c["nq"])
    return {"out": out, "lse": lse}


def _own_beam(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    c = s["case"]
    binding.beam_select(CODE[c["io"]], c["groups"], c["beams"], c["vocab"], s["logits"].data_ptr(), c["vocab"], s["scores"].data_ptr(),
                        s["weights"].data_ptr() if c["weights"] else None, s["ended"].data_ptr(), END if c["end"] else -1, c["n_out"], s["parents"].data_ptr(), s["tokens"].data_ptr(),
                        s["scores_out"].data_ptr(), s["ended_out"].data_ptr(), c["width"], s["history"].data_ptr(), s["lens"].data_ptr(), s["history_out"].data_ptr(),
                        s["lens_out"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(), s["err"].data_ptr(), torch.cuda.current_stream().cuda_stream)
    return {"parents": s["parents"], "tokens": s["tokens"], "scores": s["scores_out"], "ended": s["ended_out"], "lens": s["lens_out"], "history": s["history_out"]}


def _plain_beam(s):
    c = s["case"]
    groups, beams, vocab, n_out, width = c["groups"], c["beams"], c["vocab"], c["n_out"], c["width"]
    end = END if c["end"] else -1
    z = s["logits"].double()  # candidates of different beams may lie closer than 32 bits tell
    m = z.amax(-1, keepdim=True)
    score = s["scores"].double()[:, None] + (z - m - torch.log(torch.exp(z - m).sum(-1, keepdim=True)))
    ended = s["ended"].bool()
    score = torch.where(ended[:, None], -math.inf, score)
    kept = max(end, 0)  # an ended beam's only candidate, in the end token's place
    score[:, kept] = torch.where(ended, s["scores"].double(), score[:, kept])
    key = score * s["weights"].double()[:, None] if c["weights"] else score
    key = key.view(groups, beams * vocab)
    value, order = torch.sort(key, dim=-1, descending=True, stable=True)  # the lower index of equal ones
    value, order = value[:, :n_out], order[:, :n_out]
    alive = value > -math.inf
    row = order // vocab + torch.arange(groups, device=DEV)[:, None] * beams
    best = torch.where(alive, score.view(groups, beams * vocab).gather(1, order), -math.inf)
    old = ended[row]
    token = torch.where(old, end, order % vocab)
    parents = torch.where(alive, row, -1).view(-1)
    token = torch.where(alive, token, -1).view(-1)
    ended_out = (~alive | old | (token.view(groups, n_out) == end)).view(-1)
    length = s["lens"].long()[parents.clamp_min(0)]
    grows = (alive & ~old).view(-1)
    at = torch.arange(width, device=DEV)
    history = torch.where(at < length[:, None], s["history"][parents.clamp_min(0)], -1)
    history = torch.where(grows[:, None] & (at == length[:, None]), token.to(torch.int32)[:, None], history)
    history = torch.where((parents >= 0)[:, None], history, -1)
    lens = torch.where(parents >= 0, length + grows, 0)
    return {"parents": parents.to(torch.int32), "tokens": token.to(torch.int32), "scores": best.view(-1).float(), "ended": ended_out.to(torch.int32), "lens": lens.to(torch.int32),
            "history": history}


def _own_fork(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    c = s["case"]
    binding.page_fork(c["groups"] * c["beams"], c["groups"] * c["n_out"], c["page"], s["n_pages"], c["blocks"], s["lens"].data_ptr(), s["table"].data_ptr(), s["parents"].data_ptr(),
                      s["shares"].data_ptr(), s["free"].data_ptr(), s["n_free"].data_ptr(), s["lens_out"].data_ptr(), s["table_out"].data_ptr(), s["shares_out"].data_ptr(),
                      s["free_out"].data_ptr(), s["n_free_out"].data_ptr(), s["copy_src"].data_ptr(), s["copy_dst"].data_ptr(), s["copy_len"].data_ptr(), s["ws"].data_ptr(),
                      s["ws"].numel(), s["err"].data_ptr(), torch.cuda.current_stream().cuda_stream)
    return {"lens": s["lens_out"], "table": s["table_out"], "shares": s["shares_out"], "free": s["free_out"], "n_free": s["n_free_out"], "copy_src": s["copy_src"],
            "copy_dst": s["copy_dst"], "copy_len": s["copy_len"]}


def _plain_fork(s):
    c = s["case"]
    page, n_pages, blocks = c["page"], s["n_pages"], c["blocks"]
    n = s["lens"].shape[0]
    parents = s["parents"].long()
    there = parents >= 0
    par = parents.clamp_min(0)
    lens_in = s["lens"].long()
    lens = torch.where(there, lens_in[par], 0)
    kids = torch.zeros(n + 1, dtype=torch.int64, device=DEV).index_add_(0, torch.where(there, par, n), torch.ones_like(par))[:n]
    i = torch.arange(parents.shape[0], device=DEV)
    first = torch.full((n,), parents.shape[0], device=DEV).scatter_reduce_(0, par, torch.where(there, i, parents.shape[0]), "amin")
    takes = there & (lens % page != 0) & (i != first[par])  # gets a copy of the last page
    number = torch.cumsum(takes, 0) - takes.long()
    n_copies = takes.sum()
    n_free = s["n_free"].long()
    fresh = torch.where(takes, s["free"].long()[(n_free - 1 - number).clamp(0, n_pages - 1)], -1)
    col = torch.arange(blocks, device=DEV)
    need = (lens + page - 1) // page
    table = torch.where(col < need[:, None], s["table"][par], -1)
    last = (need - 1).clamp_min(0)[:, None]
    src = table.gather(1, last)[:, 0]
    table.scatter_(1, last, torch.where(takes, fresh.to(torch.int32), src)[:, None])
    # further holders: all of a parent's full pages gain its children but one; its last page loses its holder with the last child
    used = col < ((lens_in + page - 1) // page)[:, None]
    part = used & (col == (lens_in // page)[:, None])
    gain = torch.where(part, torch.where(kids > 0, 0, -1)[:, None], (kids - 1)[:, None])
    shares = s["shares"].long().index_add(0, s["table"][used].long(), gain[used])
    gone = shares < 0
    shares = torch.where(gone, 0, shares)
    back = gone.nonzero()[:, 0]
    keep = n_free - n_copies
    at = torch.arange(n_pages, device=DEV)
    free = torch.where(at < keep, s["free"], -1)
    free[keep + torch.arange(back.shape[0], device=DEV)] = back.to(torch.int32)
    return {"lens": lens.to(torch.int32), "table": table, "shares": shares.to(torch.int32), "free": free, "n_free": (keep + back.shape[0]).to(torch.int32),
            "copy_src": torch.where(takes, src, -1), "copy_dst": fresh.to(torch.int32), "copy_len": torch.where(takes, lens % page, 0).to(torch.int32)}


def _own_copy(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    binding.page_copy(s["kvs"], len(s["caches"]), s["case"]["n"], s["src"].data_ptr(), s["dst"].data_ptr(), s["len"].data_ptr() if s["case"]["filled"] else None, s["err"].data_ptr(),
                      torch.cuda.current_stream().cuda_stream)
    return s["caches"]


def _plain_copy(s):
    c = s["case"]
    real = (s["src"] >= 0).nonzero()[:, 0]
    src, dst = s["src"].long()[real], s["dst"].long()[real]
    for pair in s["caches"]:
        for cache in pair:
            rows = _by_position(c, cache)
            if c["filled"]:
                moved = torch.arange(c["page"], device=DEV) < s["len"][real][:, None]
                rows[dst] = torch.where(moved[:, :, None, None], rows[src], rows[dst])
            else:
                rows[dst] = rows[src]
    return s["caches"]


def _own_compact(s):
    from qwen2_decoder_forward_decode_gb300 import binding
    c = s["case"]
    binding.page_compact(c["n"], c["page"], c["pages"], c["blocks"], c["moves"], s["lens"].data_ptr(), s["table"].data_ptr(), s["shares"].data_ptr(), s["free"].data_ptr(),
                         s["n_free"].data_ptr(), s["table_out"].data_ptr(), s["shares_out"].data_ptr(), s["free_out"].data_ptr(), s["src"].data_ptr(), s["dst"].data_ptr(),
                         s["n_moves"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(), s["err"].data_ptr(), torch.cuda.current_stream().cuda_stream)
    return {"table": s["table_out"], "shares": s["shares_out"], "free": s["free_out"], "src": s["src"], "dst": s["dst"], "n_moves": s["n_moves"]}


def _plain_compact(s):
    c = s["case"]
    n_pages, most = c["pages"], c["moves"]
    at = torch.arange(n_pages, device=DEV)
    is_free = torch.zeros(n_pages + 1, dtype=torch.bool, device=DEV)
    is_free[torch.where(at < s["n_free"], s["free"].long(), n_pages)] = True
    is_free = is_free[:-1]
    live = n_pages - s["n_free"].long()
    hole = is_free & (at < live)
    high = ~is_free & (at >= live)
    hole_no = torch.cumsum(hole, 0) - 1  # from below
    high_no = torch.cumsum(high.flip(0), 0).flip(0) - 1  # from above
    n_moves = hole.sum().clamp_max(most)
    moved, filled = high & (high_no < n_moves), hole & (hole_no < n_moves)
    src = torch.full((most + 1,), -1, dtype=torch.int64, device=DEV)
    dst = src.clone()
    src[torch.where(moved, high_no, most)] = at
    dst[torch.where(filled, hole_no, most)] = at
    src, dst = src[:most], dst[:most]
    to = torch.where(moved, dst[high_no.clamp(0, most - 1)], at)
    need = (s["lens"].long() + c["page"] - 1) // c["page"]
    used = torch.arange(c["blocks"], device=DEV) < need[:, None]
    table = torch.where(used, to[s["table"].long().clamp_min(0)].to(torch.int32), s["table"])
    shares = s["shares"].clone()
    shares[at[filled]] = s["shares"][src[hole_no[filled]]]
    shares[at[moved]] = 0
    now_free = (is_free & ~filled) | moved
    free = torch.cat([at[now_free].flip(0).to(torch.int32), torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)])[:n_pages]
    return {"table": table, "shares": shares, "free": free, "src": src.to(torch.int32), "dst": dst.to(torch.int32), "n_moves": n_moves.to(torch.int32).view(1)}


# ---- the definitions in 64 bits ----------------------------------------------------------------------


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"shared": _exact_shared, "beam": _exact_beam, "fork": _exact_fork, "copy": _exact_copy, "compact": _exact_compact}[case["op"]](case, s)


def _exact_shared(c, s):
    """Every sequence by itself, over its own table."""
    grp, page = c["nq"] // c["nkv"], c["page"]
    lens = s["lens"].tolist()
    out = torch.zeros(len(lens), c["nq"], c["hd"], dtype=torch.float64, device=DEV)
    lse = torch.full((len(lens), c["nq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b, length in enumerate(lens):
        if not length:
            continue
        rows = s["table"][b, :-(-length // page)].long()
        k, v = (_by_position(c, x)[rows].reshape(-1, c["nkv"], c["hd"])[:length].double() for x in (s["kc"], s["vc"]))
        z = torch.einsum("ghd,pgd->ghp", s["q"][b].double().view(c["nkv"], grp, c["hd"]), k) / math.sqrt(c["hd"])
        lse[b] = torch.logsumexp(z, -1).view(-1)
        out[b] = torch.einsum("ghp,pgd->ghd", torch.softmax(z, -1), v).reshape(c["nq"], c["hd"])
    return {"out": out, "lse": lse}


def _exact_beam(c, s):
    groups, beams, n_out, width, end = c["groups"], c["beams"], c["n_out"], c["width"], END if c["end"] else -1
    k = groups * n_out
    parents, tokens, ended_out, lens_out = (np.full(k, v, dtype=np.int32) for v in (-1, -1, 1, 0))
    scores, history = np.full(k, -np.inf), np.full((k, width), -1, dtype=np.int32)
    c_in, ended, lens, old = s["scores"].tolist(), s["ended"].tolist(), s["lens"].tolist(), s["history"].cpu().numpy()
    weights = s["weights"].tolist() if c["weights"] else [1.0] * (groups * beams)
    for g in range(groups):
        found = []  # (-weighted score, beam, token, score)
        for w in range(g * beams, (g + 1) * beams):
            if c_in[w] == -math.inf:
                continue
            if ended[w]:
                found.append((-weights[w] * c_in[w], w, end, c_in[w]))
                continue
            lp = torch.log_softmax(s["logits"][w].double(), -1)
            least = torch.topk(lp, min(n_out, c["vocab"])).values[-1]
            for t in (lp >= least).nonzero()[:, 0].tolist():
                v = c_in[w] + float(lp[t])
                if v > -math.inf:
                    found.append((-weights[w] * v, w, t, v))
        for i, (_, w, t, v) in enumerate(sorted(found)[:n_out]):
            i += g * n_out
            parents[i], tokens[i], scores[i], ended_out[i] = w, t, v, bool(ended[w] or t == end)
            line = old[w, :lens[w]].tolist() + ([] if ended[w] else [t])
            lens_out[i] = len(line)
            history[i, :len(line)] = line
    return {"parents": parents, "tokens": tokens, "scores": scores, "ended": ended_out, "lens": lens_out, "history": history}


def _exact_fork(c, s):
    """One child after the other, holders counted in a list."""
    page, lens, table = c["page"], s["lens"].tolist(), s["table"].cpu().numpy()
    holders = np.zeros(s["n_pages"], dtype=np.int64)
    free = s["free"].tolist()[:int(s["n_free"])]
    for b, length in enumerate(lens):
        holders[table[b, :-(-length // page)]] = 1
    holders += s["shares"].cpu().numpy()
    was = holders > 0
    for b, length in enumerate(lens):
        holders[table[b, :-(-length // page)]] -= 1
    k = s["parents"].shape[0]
    out = np.full((k, c["blocks"]), -1, dtype=np.int32)
    new, src, dst, count = (np.full(k, v, dtype=np.int32) for v in (0, -1, -1, 0))
    kept = set()
    for i, p in enumerate(s["parents"].tolist()):
        if p < 0:
            continue
        new[i] = lens[p]
        pages = table[p, :-(-lens[p] // page)].copy()
        if lens[p] % page and p in kept:
            src[i], count[i] = pages[-1], lens[p] % page
            dst[i] = pages[-1] = free.pop()
        kept.add(p)
        out[i, :len(pages)] = pages
        holders[pages] += 1
    free += np.flatnonzero(was & (holders == 0)).tolist()
    rest = np.full(s["n_pages"], -1, dtype=np.int32)
    rest[:len(free)] = free
    return {"lens": new, "table": out, "shares": np.maximum(holders - 1, 0).astype(np.int32), "free": rest, "n_free": np.array([len(free)], dtype=np.int32), "copy_src": src,
            "copy_dst": dst, "copy_len": count}


def _exact_copy(c, s):
    src, dst = s["src"].tolist(), s["dst"].tolist()
    count = s["len"].tolist() if c["filled"] else [c["page"]] * c["n"]
    caches = [[_by_position(c, x).double() for x in pair] for pair in s["caches"]]
    for pair in caches:
        for rows in pair:
            for a, b, m in zip(src, dst, count):
                if a >= 0:
                    rows[b, :m] = rows[a, :m]
    return [[x.transpose(1, 2) if c["layout"] == "head" else x for x in pair] for pair in caches]


def _exact_compact(c, s):
    n_free = int(s["n_free"])
    free = set(s["free"].tolist()[:n_free])
    live = c["pages"] - n_free
    holes = sorted(p for p in free if p < live)
    high = [p for p in range(c["pages"] - 1, live - 1, -1) if p not in free]
    pairs = list(zip(high, holes))[:c["moves"]]
    shares, table = s["shares"].cpu().numpy().copy(), s["table"].cpu().numpy().copy()
    to = np.arange(c["pages"])
    for a, b in pairs:
        to[a], shares[b] = b, shares[a]
        shares[a] = 0
        free.remove(b)
        free.add(a)
    for b, length in enumerate(s["lens"].tolist()):
        k = -(-length // c["page"])
        table[b, :k] = to[table[b, :k]]
    src, dst, rest = (np.full(m, -1, dtype=np.int32) for m in (c["moves"], c["moves"], c["pages"]))
    src[:len(pairs)], dst[:len(pairs)] = [a for a, _ in pairs], [b for _, b in pairs]
    rest[:n_free] = sorted(free, reverse=True)
    return {"table": table, "shares": shares, "free": rest, "src": src, "dst": dst, "n_moves": np.array([len(pairs)], dtype=np.int32)}


# ---- what a pass cannot do without -------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "shared":
        size, _, pre, lens = _groups(c)
        own_part = np.maximum(0, lens - np.repeat(pre, size))
        total = int(pre.sum() + own_part.sum())
        rows = len(lens)
        kv = 2 * total * c["nkv"] * c["hd"] * SIZE[c["cache"]]
        ends = 2 * rows * c["nq"] * c["hd"] * SIZE[c["io"]] + 4 * rows * (c["nq"] + 2)
        return {"bytes": kv + ends + 4 * (total // c["page"]), "flops": 4 * c["nq"] * c["hd"] * int(lens.sum())}
    if c["op"] == "beam":
        rows, k = c["groups"] * c["beams"], c["groups"] * c["n_out"]
        alive = rows * 3 // 4 if c["end"] and not c["first"] else c["groups"] if c["first"] else rows  # about a quarter has ended
        return {"bytes": alive * c["vocab"] * SIZE[c["io"]] + 16 * rows + 20 * k + 4 * k * c["width"], "flops": 5 * alive * c["vocab"]}
    if c["op"] == "fork":
        n, k = c["groups"] * c["beams"], c["groups"] * c["n_out"]
        lens = _spread(4, c["groups"], c["pre_lo"], c["pre_hi"]) + _spread(5, c["groups"], c["own_lo"], c["own_hi"])
        pages = -(-lens // c["page"])
        if c["idle"]:
            pages = np.delete(pages, np.s_[3::8])
        return {"bytes": 4 * int(pages.sum()) * (c["beams"] + c["n_out"]) + 16 * int(pages.sum()) + 4 * n + 24 * k, "flops": 0}
    if c["op"] == "copy":
        count = np.random.default_rng([6, c["n"]]).integers(1, c["page"] + 1, c["n"]) if c["filled"] else np.full(c["n"], c["page"])
        moved = int(count.sum() - count[7::16].sum())
        return {"bytes": 4 * moved * c["layers"] * c["nkv"] * c["hd"] * SIZE[c["cache"]] + 12 * c["n"], "flops": 0}
    need = _spread(7, c["n"], 0, min(c["blocks"], int(2 * c["live"] * c["pages"] / c["n"])))
    return {"bytes": 8 * int(need.sum()) + 8 * c["pages"] + 8 * int((1 - c["live"]) * c["pages"]) + 8 * c["moves"], "flops": 0}
