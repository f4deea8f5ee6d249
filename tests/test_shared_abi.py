"""Refusals of the operators for continuations that share a prompt: no GPU needed. Every call here must be
turned down before anything is launched."""
import math

import pytest

import __graft_entry__
from qwen2_decoder_forward_decode_gb300 import binding


@pytest.fixture(scope="module", autouse=True)
def L():
    __graft_entry__.build()
    return binding.lib()


P = 1 << 20  # a 16-byte aligned address that is never read


def refused(call, status, word=""):
    with pytest.raises(binding.QwError) as e:
        call()
    assert e.value.status == status and word in str(e.value), str(e.value)


def cache(**over):
    c = dict(k=P, v=P, dtype=2, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, page_stride=2048, head_stride=1024, pos_stride=64)
    c.update(over)
    return binding.PagedKV(*c.values())


def attn(kv=None, **over):
    a = dict(n_seqs=4, n_heads=4, table=P, max_blocks=4, lens=P, n_groups=2, cu=P, shared=P, io=2, q=P, q_stride=256, scale=0.125, out=P + 65536, out_stride=256, lse=P, ws=P, ws_bytes=1 << 40, err=P)
    a.update(over)
    binding.shared_attention(kv or cache(), *a.values())


def beam(**over):
    a = dict(dtype=0, groups=2, beams=3, vocab=100, logits=P, stride=100, scores=P, weights=P, ended=P, end_id=1, n_out=4, parents=P, tokens=P, scores_out=P + 4096, ended_out=P + 4096, width=8, history=P,
             lens=P, history_out=P + 4096, lens_out=P + 4096, ws=P, ws_bytes=1 << 30, err=P)
    a.update(over)
    binding.beam_select(*a.values())


def fork(**over):
    a = dict(n=2, n_out=3, page=16, n_pages=8, blocks=4, lens=P, table=P, parents=P, shares=P, free=P, n_free=P, lens_out=P + 4096, table_out=P + 4096, shares_out=P, free_out=P, n_free_out=P, src=P,
             dst=P, count=P, ws=P, ws_bytes=1 << 30, err=P)
    a.update(over)
    binding.page_fork(*a.values())


def compact(**over):
    a = dict(n=2, page=16, n_pages=8, blocks=4, moves=8, lens=P, table=P, shares=P, free=P, n_free=P, table_out=P, shares_out=P, free_out=P, src=P, dst=P, n_moves=P, ws=P, ws_bytes=1 << 30, err=P)
    a.update(over)
    binding.page_compact(*a.values())


def copy(kvs=None, n_caches=2, **over):
    a = dict(n=2, src=P, dst=P, count=P, err=P)
    a.update(over)
    binding.page_copy(binding.paged_kv_array([cache()] * 2) if kvs is None else kvs, n_caches, *a.values())


@pytest.mark.parametrize("over,status,word", [
    (dict(n_seqs=-1), 1, ""), (dict(n_heads=5), 1, ""), (dict(max_blocks=0), 1, ""), (dict(io=1), 2, "io dtype"), (dict(table=None), 1, "null"), (dict(lens=None), 1, "null"), (dict(n_groups=-1), 1, "n_groups"),
    (dict(n_groups=5), 1, "n_groups"), (dict(n_groups=0), 1, "group"), (dict(cu=None), 1, "null"), (dict(shared=None), 1, "null"), (dict(q=None), 1, "null"), (dict(out=None), 1, "null"), (dict(ws=None), 1, "null"),
    (dict(err=None), 1, "null"), (dict(q_stride=128), 1, "q"), (dict(out_stride=250), 1, "out"), (dict(scale=math.nan), 1, "scale"), (dict(scale=math.inf), 1, "scale"), (dict(ws=P + 8), 1, "aligned"),
    (dict(ws_bytes=1 << 20), 1, "small"), (dict(n_seqs=65536), 2, "65535"), (dict(max_blocks=1 << 28), 2, "max_blocks"), (dict(out=P, out_stride=512), 1, "same stride"), (dict(n_seqs=60000, max_blocks=1 << 16), 2, "too large"),
])
def test_shared_attention_refusals(over, status, word):
    refused(lambda: attn(**over), status, word)


def test_shared_attention_refuses_bad_caches():
    refused(lambda: attn(cache(head_dim=60)), 2, "head_dim")
    refused(lambda: attn(cache(page_stride=1024)), 1, "overlap")
    refused(lambda: attn(cache(k=None)), 1, "null")


@pytest.mark.parametrize("over,status,word", [
    (dict(dtype=3), 1, "dtype"), (dict(groups=-1), 1, ""), (dict(beams=0), 1, ""), (dict(vocab=0), 1, ""), (dict(n_out=0), 1, ""), (dict(beams=33), 2, "32"), (dict(n_out=33), 2, "32"), (dict(groups=65536), 2, ""),
    (dict(vocab=(1 << 21) + 1, stride=1 << 22), 2, "2^21"), (dict(stride=99), 1, "overlap"), (dict(end_id=100), 1, "end_id"), (dict(end_id=-2), 1, "end_id"), (dict(history=None), 1, "all or none"),
    (dict(lens=None), 1, "all or none"), (dict(history_out=None), 1, "all or none"), (dict(lens_out=None), 1, "all or none"), (dict(width=0), 1, "width"), (dict(history_out=P), 1, "old"), (dict(lens_out=P), 1, "old"),
    (dict(scores_out=P), 1, "old"), (dict(ended_out=P), 1, "old"), (dict(logits=None), 1, "null"), (dict(scores=None), 1, "null"), (dict(parents=None), 1, "null"), (dict(tokens=None), 1, "null"),
    (dict(scores_out=None), 1, "null"), (dict(ws=None), 1, "null"), (dict(err=None), 1, "null"), (dict(ws=P + 4), 1, "aligned"), (dict(ws_bytes=0), 1, "small"), (dict(logits=P + 2), 1, "misaligned"),
])
def test_beam_refusals(over, status, word):
    refused(lambda: beam(**over), status, word)


@pytest.mark.parametrize("over,status,word", [
    (dict(n=-1), 1, ""), (dict(n_out=-1), 1, ""), (dict(page=0), 1, ""), (dict(n_pages=0), 1, ""), (dict(blocks=0), 1, ""), (dict(n=16385), 2, "16384"), (dict(n_out=16385), 2, "16384"),
    (dict(n_pages=(1 << 30) + 1), 2, "2^30"), (dict(n=16384, blocks=1 << 30), 2, "too large"), (dict(lens=None), 1, "null"), (dict(table=None), 1, "null"), (dict(parents=None), 1, "null"), (dict(shares=None), 1, "null"),
    (dict(free=None), 1, "null"), (dict(n_free=None), 1, "null"), (dict(lens_out=None), 1, "null"), (dict(table_out=None), 1, "null"), (dict(shares_out=None), 1, "null"), (dict(free_out=None), 1, "null"),
    (dict(n_free_out=None), 1, "null"), (dict(src=None), 1, "null"), (dict(dst=None), 1, "null"), (dict(count=None), 1, "null"), (dict(ws=None), 1, "null"), (dict(err=None), 1, "null"), (dict(lens_out=P), 1, "old"),
    (dict(table_out=P), 1, "old"), (dict(ws=P + 8), 1, "aligned"), (dict(ws_bytes=100), 1, "small"),
])
def test_fork_refusals(over, status, word):
    refused(lambda: fork(**over), status, word)


@pytest.mark.parametrize("over,status,word", [
    (dict(n=-1), 1, ""), (dict(page=0), 1, ""), (dict(n_pages=0), 1, ""), (dict(blocks=0), 1, ""), (dict(moves=-1), 1, ""), (dict(n_pages=(1 << 30) + 1), 2, "2^30"), (dict(moves=(1 << 30) + 1), 2, "2^30"),
    (dict(n=1 << 30, blocks=1 << 20), 2, "too large"), (dict(lens=None), 1, "null"), (dict(table=None), 1, "null"), (dict(shares=None), 1, "both"), (dict(shares_out=None), 1, "both"), (dict(free=None), 1, "null"),
    (dict(n_free=None), 1, "null"), (dict(table_out=None), 1, "null"), (dict(free_out=None), 1, "null"), (dict(src=None), 1, "null"), (dict(dst=None), 1, "null"), (dict(n_moves=None), 1, "null"),
    (dict(ws=None), 1, "null"), (dict(err=None), 1, "null"), (dict(ws=P + 8), 1, "aligned"), (dict(ws_bytes=100), 1, "small"),
])
def test_compact_refusals(over, status, word):
    refused(lambda: compact(**over), status, word)


def test_copy_refusals():
    refused(lambda: copy(n_caches=-1), 1)
    refused(lambda: copy(n=-1), 1)
    refused(lambda: copy(binding.paged_kv_array([cache()] * 129), 129), 2, "128")
    refused(lambda: binding.page_copy(None, 2, 2, P, P, None, P), 1, "null")
    refused(lambda: copy(binding.paged_kv_array([cache(), cache(v=None)])), 1, "null")
    refused(lambda: copy(binding.paged_kv_array([cache(), cache(head_dim=60)])), 2, "head_dim")
    for other in (dict(dtype=1), dict(n_pages=9), dict(page_size=8), dict(n_kv_heads=1), dict(head_dim=32), dict(page_stride=4096), dict(pos_stride=128, head_stride=2048, page_stride=4096)):
        refused(lambda: copy(binding.paged_kv_array([cache(), cache(**other)])), 2, "same type")
    for name in ("src", "dst", "err"):
        refused(lambda: copy(**{name: None}), 1, "null")


def test_nothing_to_do_is_no_error():
    attn(n_seqs=0, n_groups=0, q=None, table=None)
    beam(groups=0, logits=None)
    copy(n=0, src=None)
    copy(n_caches=0, src=None)


@pytest.mark.parametrize("call,names", [
    (attn, ("table", "lens", "cu", "shared", "lse", "err")), (beam, ("scores", "weights", "ended", "parents", "tokens", "scores_out", "ended_out", "history", "lens", "history_out", "lens_out", "err")),
    (fork, ("lens", "table", "parents", "shares", "free", "n_free", "lens_out", "table_out", "shares_out", "free_out", "n_free_out", "src", "dst", "count", "err")),
    (compact, ("lens", "table", "shares", "free", "n_free", "table_out", "shares_out", "free_out", "src", "dst", "n_moves", "err")), (copy, ("src", "dst", "count", "err")),
])
def test_pointers_between_two_elements_are_refused(call, names):
    for name in names:
        for off in (1, 2, 3):
            refused(lambda: call(**{name: P + 8192 + off}), 1, "aligned")


def test_workspace_sizes(L):
    assert L.qw_op_shared_attention_workspace(4, 12, 2, 128) > L.qw_op_paged_attention_workspace(12, 2, 128)
    assert L.qw_op_shared_attention_workspace(4, 12, 5, 128) == 0 and L.qw_op_shared_attention_workspace(65536, 12, 2, 128) == 0
    # states of both parts for every sequence and head, and 320 tiles of 128 rows (or 640 of 64), with m and l in a row of 4 more
    for hd, pad in ((8, 64), (64, 64), (96, 128), (128, 128)):
        assert L.qw_op_shared_attention_workspace(300, 12, 2, hd) >= 2 * 300 * 12 * (hd + 4) * 4 + 320 * 128 * (pad + 4) * 4
    assert L.qw_op_shared_attention_workspace(300, 12, 2, 256) >= 2 * 300 * 12 * 260 * 4 + 320 * 64 * 260 * 4
    assert L.qw_op_beam_select_workspace(2, 4, 1000, 8) > 0 and L.qw_op_beam_select_workspace(2, 33, 1000, 8) == 0
    assert L.qw_op_page_fork_workspace(100) >= 400 and L.qw_op_page_fork_workspace(0) == 0
    assert L.qw_op_page_compact_workspace(100) >= 400 and L.qw_op_page_compact_workspace(0) == 0
