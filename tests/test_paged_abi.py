"""Refusals of the paged-cache operators and the host-side rotary frequencies: no GPU needed. Every
call here must be turned down before anything is launched."""
import ctypes
import math

import numpy as np
import pytest

import __graft_entry__
from qwen2_decoder_forward_decode_gb300 import binding


@pytest.fixture(scope="module", autouse=True)
def L():
    __graft_entry__.build()
    return binding.lib()


P = 1 << 20  # a 16-byte aligned address that is never read


def cache(**over):
    c = dict(k=P, v=P, dtype=2, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, page_stride=2048, head_stride=1024, pos_stride=64)
    c.update(over)
    return binding.PagedKV(*c.values())


def refused(call, status, word=""):
    with pytest.raises(binding.QwError) as e:
        call()
    assert e.value.status == status and word in str(e.value), str(e.value)


BAD_CACHES = [
    (dict(k=None), 1, "null"), (dict(v=None), 1, "null"), (dict(dtype=7), 1, "dtype"), (dict(n_pages=0), 1, ""), (dict(page_size=0), 1, ""), (dict(n_kv_heads=0), 1, ""),
    (dict(head_dim=0), 1, ""), (dict(head_dim=60), 2, "head_dim"), (dict(head_dim=264), 2, "head_dim"), (dict(k=P + 8), 1, "aligned"), (dict(v=P + 2), 1, "aligned"),
    (dict(pos_stride=68), 1, "16 bytes"), (dict(page_stride=-2048), 1, "stride"), (dict(pos_stride=56), 1, "overlap"), (dict(head_stride=512), 1, "overlap"),
    (dict(page_stride=1024), 1, "overlap"), (dict(page_stride=64, pos_stride=2048, head_stride=32768), 1, "overlap"), (dict(page_stride=1 << 50), 1, "stride"),
]


def attn(kv=None, **over):
    a = dict(n_seqs=2, n_heads=4, table=P, max_blocks=4, lens=P, io=2, q=P, q_stride=256, scale=0.125, out=P + 65536, out_stride=256, lse=P, ws=P, ws_bytes=1 << 30, err=P)
    a.update(over)
    binding.paged_attention(kv or cache(), *a.values())


def rope(kv=None, **over):
    a = dict(n_tokens=2, n_heads=4, io=2, positions=P, slots=P, turns=P, rot=64, adjacent=0, mscale=1.0, q=P, qs=256, k=P, ks=128, v=P, vs=128, q_out=P, qos=256, err=P)
    a.update(over)
    binding.rope_append(kv or cache(), *a.values())


@pytest.mark.parametrize("over,status,word", BAD_CACHES)
def test_bad_caches_are_refused(over, status, word):
    refused(lambda: attn(cache(**over)), status, word)
    refused(lambda: rope(cache(**over)), status, word)


@pytest.mark.parametrize("over,status,word", [
    (dict(n_seqs=-1), 1, ""), (dict(n_heads=5), 1, ""), (dict(n_heads=0), 1, ""), (dict(max_blocks=0), 1, ""), (dict(io=1), 2, "io dtype"), (dict(io=9), 1, "dtype"), (dict(table=None), 1, "null"),
    (dict(lens=None), 1, "null"), (dict(q=None), 1, "null"), (dict(out=None), 1, "null"), (dict(ws=None), 1, "null"), (dict(err=None), 1, "null"), (dict(q=P + 4), 1, "q"), (dict(q_stride=250), 1, "q"),
    (dict(q_stride=128), 1, "q"), (dict(out_stride=128), 1, "out"), (dict(scale=math.inf), 1, "scale"), (dict(scale=math.nan), 1, "scale"), (dict(ws=P + 8), 1, "aligned"), (dict(ws_bytes=16), 1, "small"),
    (dict(n_seqs=65536), 2, "65535"), (dict(max_blocks=1 << 28), 2, "max_blocks"), (dict(out=P, out_stride=512), 1, "same stride"), (dict(n_heads=8192), 2, "4096"),
])
def test_attention_refusals(over, status, word):
    refused(lambda: attn(**over), status, word)


@pytest.mark.parametrize("over,status,word", [
    (dict(n_tokens=-1), 1, ""), (dict(n_heads=0), 1, ""), (dict(io=1), 2, "io dtype"), (dict(rot=0), 1, "rot_dim"), (dict(rot=63), 1, "rot_dim"), (dict(rot=66), 1, "rot_dim"), (dict(adjacent=2), 1, "adjacent"),
    (dict(mscale=math.nan), 1, "mscale"), (dict(positions=None), 1, "null"), (dict(slots=None), 1, "null"), (dict(turns=None), 1, "null"), (dict(slots=P + 4), 1, "aligned"), (dict(turns=P + 4), 1, "aligned"),
    (dict(q=P + 8), 1, "q"), (dict(k=None), 1, "null"), (dict(ks=64), 1, "k"), (dict(vs=132), 1, "v"), (dict(qos=512), 1, "same stride"), (dict(err=None), 1, "null"), (dict(q_out=None), 1, "null"),
])
def test_rope_refusals(over, status, word):
    refused(lambda: rope(**over), status, word)


def plan(**over):
    a = dict(n=2, page=16, n_pages=8, blocks=4, tokens=8, lens=P, new=P, free=P, n_free=P, table=P, lens_out=P, n_free_out=P, cu=P, positions=P, slots=P, err=P)
    a.update(over)
    binding.page_plan(*a.values())


def release(**over):
    a = dict(n=2, page=16, n_pages=8, blocks=4, lens=P, done=P, table=P, free=P, n_free=P, lens_out=P, n_free_out=P, err=P)
    a.update(over)
    binding.page_release(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), 1), (dict(page=0), 1), (dict(n_pages=0), 1), (dict(blocks=0), 1), (dict(n=16385), 2), (dict(lens=None), 1), (dict(free=None), 1), (dict(n_free=None), 1), (dict(table=None), 1),
    (dict(lens_out=None), 1), (dict(n_free_out=None), 1), (dict(err=None), 1),
])
def test_plan_and_release_refusals(over, status):
    refused(lambda: plan(**over), status)
    refused(lambda: release(**over), status)


@pytest.mark.parametrize("over", [dict(tokens=-1), dict(cu=None), dict(positions=None), dict(slots=None), dict(slots=P + 4)])
def test_plan_refusals(over):
    refused(lambda: plan(**over), 1)


def test_sizes_beyond_32_bits_are_refused():
    refused(lambda: plan(tokens=(1 << 30) + 1), 2)
    refused(lambda: plan(n_pages=(1 << 30) + 1), 2)
    refused(lambda: release(n_pages=(1 << 30) + 1), 2)
    refused(lambda: rope(n_tokens=(1 << 30) + 1), 2)
    refused(lambda: attn(n_seqs=60000, max_blocks=1 << 16), 2, "too large")
    refused(lambda: logprobs(rows=1 << 20, vocab=1 << 24, stride=1 << 24), 2, "too large")


def test_tile_lists_beyond_31_bits_are_refused():
    """Tables that share pages can hold any lengths. Tiles have 16 positions in fp32 caches of more than 128
    dimensions, at least 32 else: the same shape is within the range there."""
    def status(dtype, hd, n_seqs):
        kv = cache(dtype=dtype, head_dim=hd, n_kv_heads=1, page_stride=16 * hd, head_stride=0, pos_stride=hd)
        with pytest.raises(binding.QwError) as e:  # (in range: refused for its addresses, or for want of a GPU)
            attn(kv, n_seqs=n_seqs, n_heads=63, max_blocks=1 << 16, io=dtype, q_stride=63 * hd, out_stride=63 * hd)
        return e.value.status, str(e.value)
    for hd in (136, 256):
        assert status(0, hd, 1024)[0] == 2 and "too large" in status(0, hd, 1024)[1]
        assert status(0, hd, 521)[0] == 2 and status(0, hd, 520)[0] != 2  # 63 * 2^16 tiles: 2^31 is 520.1 times that
        assert status(2, hd, 1024)[0] != 2 and status(1, hd, 1024)[0] != 2
    assert status(0, 128, 1040)[0] != 2 and status(0, 128, 1041)[0] == 2


def test_scales_that_overflow_in_base_2_are_refused():
    for scale in (3e38, -3e38, 2.0 ** 127 * (1 + 2.0 ** -23), -math.inf):
        refused(lambda: attn(scale=scale), 1, "scale")
    for scale in (2.0 ** 127, -2.0 ** 127):
        with pytest.raises(binding.QwError) as e:  # (refused for its addresses, or for want of a GPU)
            attn(scale=scale)
        assert "scale" not in str(e.value)


def test_release_refuses_no_flags():
    refused(lambda: release(done=None), 1)


def logprobs(**over):
    a = dict(dtype=0, rows=2, vocab=100, logits=P, stride=100, ids=P, n_ids=1, lp=P, ranks=P, entropy=P, top=5, top_ids=P, top_lp=P, ws=P, ws_bytes=1 << 30, err=P)
    a.update(over)
    binding.token_logprobs(*a.values())


@pytest.mark.parametrize("over", [
    dict(dtype=4), dict(rows=-1), dict(vocab=0), dict(stride=99), dict(n_ids=9), dict(n_ids=-1), dict(top=33), dict(top=-1), dict(vocab=4, top=5), dict(logits=None), dict(ids=None), dict(lp=None),
    dict(top_ids=None), dict(top_lp=None), dict(ws=None), dict(ws=P + 8), dict(ws_bytes=0), dict(err=None), dict(logits=P + 2),
])
def test_logprobs_refusals(over):
    refused(lambda: logprobs(**over), 1)


def test_nothing_to_do_is_no_error():
    attn(n_seqs=0, q=None, table=None)
    rope(n_tokens=0, q=None)
    logprobs(rows=0, logits=None)


@pytest.mark.parametrize("call,names", [
    (attn, ("table", "lens", "lse", "err")), (rope, ("positions", "err")), (logprobs, ("ids", "lp", "ranks", "entropy", "top_ids", "top_lp", "err")),
    (plan, ("lens", "new", "free", "n_free", "table", "lens_out", "n_free_out", "cu", "positions", "err")),
    (release, ("lens", "done", "table", "free", "n_free", "lens_out", "n_free_out", "err")),
])
def test_pointers_between_two_elements_are_refused(call, names):
    for name in names:
        for off in (1, 2, 3):
            refused(lambda: call(**{name: P + off}), 1, "aligned")
    with pytest.raises(binding.QwError) as e:  # 16-bit logits may begin at any of them: refused for other reasons only
        logprobs(dtype=2, logits=P + 2)
    assert "aligned" not in str(e.value)
    refused(lambda: logprobs(dtype=2, logits=P + 1), 1, "misaligned")


def test_workspace_sizes(L):
    assert L.qw_op_paged_attention_workspace(12, 2, 128) > 0
    assert L.qw_op_paged_attention_workspace(12, 5, 128) == 0
    assert L.qw_op_paged_attention_workspace(12, 2, 12) == 0
    assert L.qw_op_token_logprobs_workspace(4, 1000, 5) > 0
    assert L.qw_op_token_logprobs_workspace(4, 1000, 33) == 0


@pytest.mark.parametrize("group", [1, 4, 8, 9, 16, 40])
@pytest.mark.parametrize("hd", [8, 32, 40, 64, 96, 128, 136, 256])
def test_the_attention_workspace_holds_every_part(L, group, hd):
    """640 parts of the kernel's heads and dimensions (16-bit caches: 64 dimensions at least for groups of more than 8
    heads), each with a maximum and a sum in a row of 4 more, and the counters."""
    pad = next(x for x in (32, 64, 128, 256) if hd <= x and (x > 32 or group <= 8))
    assert L.qw_op_paged_attention_workspace(2 * group, 2, hd) >= 16384 + 640 * (16 if group > 8 else 8) * (pad + 4) * 4


def test_model_logprobs_refuses_a_null_model(L):
    assert L.qw_read_logprobs(None, 0, None, 0, None, None, None, 0, None, None) == 1


def frequencies(r, theta, scaling, factor, orig, low, high):
    """The formulas, with loops and math alone."""
    out = []
    for i in range(r // 2):
        base = theta * factor ** (r / (r - 2)) if scaling == "ntk" and r > 2 else theta
        w = base ** (-2 * i / r)
        if scaling == "linear":
            w /= factor
        if scaling == "yarn":
            at = [r * math.log(orig / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (high, low)]
            a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
            c = min(max((i - a) / max(b - a, 1e-3), 0), 1)
            w = (1 - c) * w + c * w / factor
        if scaling == "bands":
            n = orig * w / (2 * math.pi)
            c = 0 if n <= low else 1 if n >= high else (n - low) / (high - low)
            w = c * w + (1 - c) * w / factor
        out.append(w)
    return np.array(out)


@pytest.mark.parametrize("r", [2, 16, 48, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor,orig,low,high", [
    ("none", 1.0, 0, 1, 4), ("linear", 4.0, 0, 1, 4), ("ntk", 8.0, 0, 1, 4), ("yarn", 4.0, 32768, 1, 32), ("yarn", 40.0, 4096, 1, 32), ("bands", 8.0, 8192, 1, 4), ("bands", 32.0, 4096, 1, 4),
])
def test_rope_turns_match_the_formulas(r, scaling, factor, orig, low, high):
    turns, mscale = binding.rope_turns(r, 1e6, scaling, factor, orig, low, high)
    want = frequencies(r, 1e6, scaling, factor, orig, low, high)
    got = turns.astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    # pow and the blends: a few steps of 2^-53, and the cut to 2^-65 turns
    np.testing.assert_allclose(got, want, rtol=1e-13, atol=2 * math.pi * 2.0 ** -64)
    assert mscale == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0, rel=2.0 ** -23)


def test_rope_turns_defaults():
    a, _ = binding.rope_turns(64, 1e4, "yarn", 4.0, 4096)
    b, _ = binding.rope_turns(64, 1e4, "yarn", 4.0, 4096, 1.0, 32.0)
    np.testing.assert_array_equal(a, b)
    a, _ = binding.rope_turns(64, 1e4, "bands", 4.0, 4096)
    b, _ = binding.rope_turns(64, 1e4, "bands", 4.0, 4096, 1.0, 4.0)
    np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("args", [
    (0, 1e6), (7, 1e6), (-2, 1e6), (64, 1.0), (64, math.nan), (64, math.inf), (64, 1e6, "linear", 0.5), (64, 1e6, "linear", math.nan), (64, 1e6, "yarn", 4.0, 0.0), (64, 1e6, "yarn", 4.0, 4096, 0.0),
    (64, 1e6, "bands", 4.0, 4096, 4.0, 4.0), (64, 1e6, "bands", 4.0, 4096, 1.0, math.inf), (64, 1e6, "unknown"),
])
def test_rope_turns_refusals(args):
    refused(lambda: binding.rope_turns(*args), 1)


def test_rope_turns_refuses_unknown_scaling_and_null(L):
    buf = (ctypes.c_uint64 * 32)()
    m = ctypes.c_float()
    assert L.qw_rope_turns(64, 1e6, 5, 2.0, 4096.0, 1.0, 4.0, buf, ctypes.byref(m)) == 1
    assert L.qw_rope_turns(64, 1e6, 0, 2.0, 4096.0, 1.0, 4.0, None, ctypes.byref(m)) == 1
