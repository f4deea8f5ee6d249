"""Plain 64-bit implementations of the paged-cache operators, written from their formulas, and the
buffers that the GPU tests share."""
import math

import numpy as np

CODE = {"f32": 0, "bf16": 1, "f16": 2}
EPS_HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}                   # half a subnormal step
U = 2.0 ** -23  # one step of an fp32 sum (tensor cores cut instead of rounding)


def torch_dtype(t):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[t]


def pages_of(n, page):
    return -(-n // page)


def plan(lens, new, page, table, free, max_tokens):
    """free: the free pages in use order from the end. Returns table, lens, free, cu, positions, slots."""
    table, free = table.copy(), list(free)
    cu, positions, slots = [0], [], []
    for b, (length, add) in enumerate(zip(lens, new)):
        for j in range(pages_of(length, page), pages_of(length + add, page)):
            table[b, j] = free.pop()
        for p in range(length, length + add):
            positions.append(p)
            slots.append(int(table[b, p // page]) * page + p % page)
        cu.append(cu[-1] + add)
    rest = max_tokens - cu[-1]
    return table, [a + b for a, b in zip(lens, new)], free, cu, positions + [0] * rest, slots + [-1] * rest


def rope(x, pos, freqs, adjacent, mscale, rot):
    """x [T][heads][hd] float64."""
    y = x.copy()
    i = np.arange(rot // 2)
    e, f = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
    ang = np.fmod(np.asarray(pos, dtype=np.float64)[:, None] * freqs[None, :], 2 * math.pi)
    c, s = (mscale * np.cos(ang))[:, None, :], (mscale * np.sin(ang))[:, None, :]
    y[:, :, e] = x[:, :, e] * c - x[:, :, f] * s
    y[:, :, f] = x[:, :, e] * s + x[:, :, f] * c
    return y


def rope_bound(x, adjacent, mscale, rot):
    """3 * 2^-23 (|a| + |b|) mscale per rotated dimension: cos and sin are off by at most 1.5 * 2^-23
    (an angle of at most pi/4 rounded once, one step of sincospi, mscale's product), the two
    products and their sum by half a step each."""
    tol = np.zeros_like(x)
    i = np.arange(rot // 2)
    e, f = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
    both = (np.abs(x[:, :, e]) + np.abs(x[:, :, f])) * 3 * U * mscale
    tol[:, :, e] = both
    tol[:, :, f] = both
    return tol


def attention(q, k, v, scale):
    """q [g][hd], k, v [n][hd] float64 of one KV head: (out [g][hd], lse [g], bound [g][hd]).

    The bound: a score is off by ds = (8 sqrt(hd) + 4) U scale sum |q k| (rounded sums of hd products at
    8 standard deviations, operands split into two halves of 11 bits: 2^-22), every probability by a
    relative 2 ds + 4 U, and the weighted sum by 8 sqrt(n) U of sum p |v|."""
    if len(k) == 0:
        return np.zeros(q.shape), np.full(len(q), -np.inf), np.zeros(q.shape)
    with np.errstate(all="ignore"):
        z = scale * (q @ k.T)
        m = z.max(-1, keepdims=True)
        e = np.exp(z - m)
        p = e / e.sum(-1, keepdims=True)
        ds = ((8 * math.sqrt(q.shape[1]) + 4) * U * abs(scale) * (np.abs(q) @ np.abs(k).T)).max(-1, keepdims=True)
        bound = (2 * ds + 4 * U + 8 * math.sqrt(len(k)) * U) * (p @ np.abs(v))
        return p @ v, (m + np.log(e.sum(-1, keepdims=True)))[:, 0], bound


class PagedCache:
    """A torch cache of n_pages pages with the keys and values of given sequences in shuffled pages;
    every other place holds NaN."""

    def __init__(self, rng, lens, nkv, hd, page, dtype, layout="head", spare=3, gap=0, scale=1.0, blocks=None):
        import torch
        from qwen2_decoder_forward_decode_gb300 import binding
        self.lens, self.nkv, self.hd, self.page, self.dtype = list(lens), nkv, hd, page, dtype
        need = [pages_of(n, page) for n in lens]
        self.n_pages = sum(need) + spare
        self.blocks = max([1] + need) if blocks is None else blocks
        order = list(rng.permutation(self.n_pages))
        self.table = np.full((len(lens), self.blocks), 2 ** 31 - 1, dtype=np.int32)  # unused entries are no pages
        self.free = order[sum(need):]
        unit = {"f32": 4, "f16": 8, "bf16": 8}[dtype]
        shape = (self.n_pages, nkv, page, hd + gap * unit) if layout == "head" else (self.n_pages, page, nkv, hd + gap * unit)
        self.tk, self.tv = (torch.full(shape, float("nan"), dtype=torch_dtype(dtype)) for _ in range(2))
        self.k, self.v = [], []
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            kv = []
            for t in (self.tk, self.tv):
                x = torch.from_numpy(rng.standard_normal((n, nkv, hd)) * scale).to(torch_dtype(dtype))
                for j in range(need[b]):
                    rows = x[j * page:(j + 1) * page]
                    dst = t[int(self.table[b, j]), ..., :hd]
                    dst = dst.transpose(0, 1) if layout == "head" else dst
                    dst[:len(rows)] = rows
                kv.append(x.double().numpy())
            self.k.append(kv[0])
            self.v.append(kv[1])
        self.tk, self.tv = self.tk.cuda(), self.tv.cuda()
        st = self.tk.stride()
        head, pos = (st[1], st[2]) if layout == "head" else (st[2], st[1])
        self.kv = binding.PagedKV(self.tk.data_ptr(), self.tv.data_ptr(), CODE[dtype], self.n_pages, page, nkv, hd, st[0], head, pos)
        self.layout = layout
        self.ttable = torch.from_numpy(self.table).cuda()
        self.tlens = torch.tensor(self.lens, dtype=torch.int32).cuda()

    def row(self, t, slot):
        """[nkv][hd] of a slot of self.tk or self.tv."""
        page = t[slot // self.page]
        return (page[:, slot % self.page] if self.layout == "head" else page[slot % self.page])[..., :self.hd]
