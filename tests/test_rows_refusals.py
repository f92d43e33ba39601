"""The entry points of packed and tree attention and of the block tables' growth refuse what they cannot do, before anything
is launched: host only, the device addresses are never dereferenced."""

import ctypes

import pytest
import torch

import layout_permuting_copy_amd as L
from test_paged_refusals import BASE, BIG, DIM, HEADS, PAGE, PAGES, _cache, _lay, _ref

MB = 1 << 20


def _prompt(dtype=L.TC_BF16, q_shape=(30, 4, DIM), k_shape=(30, HEADS, DIM), v_shape=None, out_shape=None, q=BASE, k=BASE + 4 * MB,
            v=BASE + 8 * MB, out=BASE + 12 * MB, q_stride=None, k_stride=None, v_stride=None, out_stride=None, batch=3,
            starts=BASE + 16 * MB, key_starts=None, causal=1, scale=1.0, lse=None, lse_shape=(30, 4), lse_stride=None, offset=0,
            work=BASE + 256 * MB, work_bytes=1 << 30):
    ql, kl, vl = _lay(q_shape, q_stride, offset), _lay(k_shape, k_stride), _lay(v_shape or k_shape, v_stride)
    ol, ll = _lay(out_shape or q_shape, out_stride), _lay(lse_shape, lse_stride)
    return L.load_library().tc_prompt_attention(q, _ref(ql), k, _ref(kl), v, _ref(vl), out, _ref(ol), dtype, batch, starts, key_starts,
                                                causal, scale, lse, _ref(ll), work, work_bytes, None)


def _tree(cache=None, dtype=L.TC_BF16, q=BASE + 4 * MB, q_shape=(30, 4, DIM), q_stride=None, out=BASE + 8 * MB, out_shape=None,
          out_stride=None, table=(3, 4), lens=BASE + 16 * MB, starts=BASE + 17 * MB, masks=None, max_len=64, scale=1.0, lse=None,
          lse_shape=(30, 4), work=BASE + 256 * MB, work_bytes=1 << 30):
    cache = _cache() if cache is None else cache
    ql, ol, tl, ll = _lay(q_shape, q_stride), _lay(out_shape or q_shape, out_stride), _lay(table), _lay(lse_shape)
    return L.load_library().tc_paged_tree_attention(_ref(cache), q, _ref(ql), out, _ref(ol), dtype, BASE + 18 * MB, _ref(tl), lens, starts,
                                                    masks, max_len, scale, lse, _ref(ll), work, work_bytes, None)


def _resize(table=BASE, shape=(3, 4), stride=None, lens=BASE + MB, change=BASE + 2 * MB, page=16, free=BASE + 3 * MB, capacity=20,
            count=BASE + 4 * MB, lens_out=BASE + 5 * MB, count_out=BASE + 6 * MB, missing=None, starts=BASE + 7 * MB, slots=None,
            positions=None, tokens=0):
    tl = _lay(shape, stride)
    return L.load_library().tc_paged_resize(table, _ref(tl), lens, change, page, free, capacity, count, lens_out, count_out, missing,
                                            starts, slots, positions, tokens, None)


ROW = 4 * DIM
PROMPT = [
    (L.TC_E_DTYPE, "dtype", lambda: _prompt(dtype=L.TC_F32)),
    (L.TC_E_DTYPE, "dtype", lambda: _prompt(dtype=L.TC_E4M3)),
    (L.TC_E_EXTENT, "q and out", lambda: _prompt(out_shape=(30, 4, DIM + 16))),
    (L.TC_E_EXTENT, "k and v", lambda: _prompt(v_shape=(29, HEADS, DIM))),
    (L.TC_E_EXTENT, "head_dim", lambda: _prompt(k_shape=(30, HEADS, DIM + 16))),
    (L.TC_E_EXTENT, "head_dim", lambda: _prompt(q_shape=(30, 4, 72), k_shape=(30, HEADS, 72))),
    (L.TC_E_EXTENT, "head_dim", lambda: _prompt(q_shape=(30, 4, 272), k_shape=(30, HEADS, 272))),
    (L.TC_E_EXTENT, "head_dim", lambda: _prompt(q_shape=(30, 4, 0), k_shape=(30, HEADS, 0))),
    (L.TC_E_EXTENT, "multiple", lambda: _prompt(q_shape=(30, 3, DIM))),
    (L.TC_E_EXTENT, "multiple", lambda: _prompt(k_shape=(30, 0, DIM))),
    (L.TC_E_EXTENT, "one key", lambda: _prompt(k_shape=(31, HEADS, DIM))),
    (L.TC_E_EXTENT, "lse", lambda: _prompt(lse=BASE + 20 * MB, lse_shape=(30, 5))),
    (L.TC_E_EXTENT, "multiple", lambda: _prompt(batch=-1)),
    (L.TC_E_RANK, "q", lambda: _prompt(q_shape=(30, 4 * DIM))),
    (L.TC_E_NULL, "q", lambda: _prompt(q=None)),
    (L.TC_E_NULL, "v", lambda: _prompt(v=None)),
    (L.TC_E_NULL, "out", lambda: _prompt(out=None)),
    (L.TC_E_NULL, "token_starts", lambda: _prompt(starts=None)),
    (L.TC_E_ALIGN, "token_starts", lambda: _prompt(starts=BASE + 16 * MB + 2)),
    (L.TC_E_ALIGN, "q: rows", lambda: _prompt(q=BASE + 8)),
    (L.TC_E_ALIGN, "q: rows", lambda: _prompt(offset=4)),
    (L.TC_E_ALIGN, "k: rows", lambda: _prompt(k_stride=(2 * DIM + 4, DIM, 1))),
    (L.TC_E_ALIGN, "v: rows", lambda: _prompt(v_stride=(2 * DIM + 8, DIM + 4, 1))),
    (L.TC_E_ALIGN, "out: rows", lambda: _prompt(out=BASE + 12 * MB + 4)),
    (L.TC_E_ARG, "innermost", lambda: _prompt(q_stride=(2 * ROW, 2 * DIM, 2))),
    (L.TC_E_ARG, "innermost", lambda: _prompt(k_stride=(2 * ROW, 2 * DIM, 2))),
    (L.TC_E_ARG, "negative", lambda: _prompt(v_stride=(-2 * DIM, DIM, 1))),
    (L.TC_E_ARG, "causal", lambda: _prompt(causal=2)),
    (L.TC_E_ARG, "scale", lambda: _prompt(scale=float("nan"))),
    (L.TC_E_ARG, "scale", lambda: _prompt(scale=float("inf"))),
    (L.TC_E_ARG, "scale", lambda: _prompt(scale=3e38)),
    (L.TC_E_NONINJECTIVE, "out", lambda: _prompt(out_stride=(0, DIM, 1))),
    (L.TC_E_NONINJECTIVE, "lse", lambda: _prompt(lse=BASE + 20 * MB, lse_stride=(1, 1))),
    (L.TC_E_ALIAS, "an output", lambda: _prompt(out=BASE)),
    (L.TC_E_ALIAS, "an output", lambda: _prompt(out=BASE + 4 * MB + 64)),
    (L.TC_E_ALIAS, "an output", lambda: _prompt(lse=BASE + 8 * MB)),
    (L.TC_E_ALIAS, "an output", lambda: _prompt(out=BASE + 16 * MB)),
    (L.TC_E_ALIAS, "an output", lambda: _prompt(key_starts=BASE + 12 * MB)),
    (L.TC_E_ALIAS, "two outputs", lambda: _prompt(lse=BASE + 12 * MB)),
    (L.TC_E_RANGE, "2^24", lambda: _prompt(k_stride=(1 << 23, DIM, 1), out=BASE + (1 << 36))),
    (L.TC_E_RANGE, "2^24", lambda: _prompt(v_stride=(1 << 23, DIM, 1), out=BASE + (1 << 36))),
    (L.TC_E_RANGE, "2^58", lambda: _prompt(q_stride=(BIG, DIM, 1))),
    (L.TC_E_RANGE, "2^30", lambda: _prompt(q_shape=(1 << 29, 4, 16), k_shape=(1 << 29, 2, 16), out_shape=(1 << 29, 4, 16))),
    (L.TC_E_RANGE, "65535", lambda: _prompt(q_shape=(1, 65536, 16), k_shape=(1, 1, 16))),
    (L.TC_E_ARG, "workspace", lambda: _prompt(k_shape=(6000, HEADS, DIM), key_starts=BASE + 17 * MB, work_bytes=0)),
    (L.TC_E_NULL, "workspace", lambda: _prompt(k_shape=(6000, HEADS, DIM), key_starts=BASE + 17 * MB, work=None)),
    (L.TC_E_ALIGN, "workspace", lambda: _prompt(k_shape=(6000, HEADS, DIM), key_starts=BASE + 17 * MB, work=BASE + 256 * MB + 4)),
    (L.TC_E_ALIAS, "an output", lambda: _prompt(k_shape=(6000, HEADS, DIM), key_starts=BASE + 17 * MB, work=BASE)),
    (L.TC_E_ALIAS, "two outputs", lambda: _prompt(k_shape=(6000, HEADS, DIM), key_starts=BASE + 17 * MB, work=BASE + 12 * MB)),
    (L.TC_E_RANGE, "keys", lambda: _prompt(q_shape=(1, 1, 16), k_shape=((1 << 30) + 1, 1, 16), key_starts=BASE + 17 * MB)),
]
TREE = [
    (L.TC_E_NULL, "null cache", lambda: L.load_library().tc_paged_tree_attention(None, 1, None, 1, None, L.TC_BF16, 1, None, 1, 1, None, 1, 1.0,
                                                                              None, None, None, 0, None)),
    (L.TC_E_DTYPE, "dtype", lambda: _tree(dtype=L.TC_F32)),
    (L.TC_E_DTYPE, "differ in type", lambda: _tree(dtype=L.TC_F16)),
    (L.TC_E_DTYPE, "dtype", lambda: _tree(_cache(dtype=L.TC_F32))),
    (L.TC_E_EXTENT, "head_dim", lambda: _tree(q_shape=(30, 4, 80))),
    (L.TC_E_EXTENT, "multiple", lambda: _tree(q_shape=(30, 3, DIM))),
    (L.TC_E_EXTENT, "q and out", lambda: _tree(out_shape=(29, 4, DIM))),
    (L.TC_E_EXTENT, "lse", lambda: _tree(lse=BASE + 20 * MB, lse_shape=(3, 4))),
    (L.TC_E_RANK, "block_table", lambda: _tree(table=(3,))),
    (L.TC_E_NULL, "seq_lens", lambda: _tree(lens=None)),
    (L.TC_E_NULL, "token_starts", lambda: _tree(starts=None)),
    (L.TC_E_ALIGN, "masks", lambda: _tree(masks=BASE + 19 * MB + 4)),
    (L.TC_E_ALIGN, "q: rows", lambda: _tree(q=BASE + 4 * MB + 2)),
    (L.TC_E_ALIGN, "out: rows", lambda: _tree(out_stride=(4 * DIM + 4, DIM, 1))),
    (L.TC_E_ALIGN, "workspace", lambda: _tree(max_len=5000, work=BASE + 256 * MB + 8)),
    (L.TC_E_ARG, "scale", lambda: _tree(scale=float("nan"))),
    (L.TC_E_ARG, "workspace", lambda: _tree(max_len=5000, work_bytes=64)),
    (L.TC_E_NULL, "workspace", lambda: _tree(max_len=5000, work=None)),
    (L.TC_E_RANGE, "max_len", lambda: _tree(max_len=(1 << 30) + 1)),
    (L.TC_E_RANGE, "max_len", lambda: _tree(max_len=-1)),
    (L.TC_E_RANGE, "2^30", lambda: _tree(_cache(shape=(PAGES, PAGE, 2, 16)), q_shape=(1 << 29, 4, 16), out=BASE + (1 << 40))),
    (L.TC_E_ALIAS, "the cache", lambda: _tree(out=BASE + 64)),
    (L.TC_E_ALIAS, "the cache", lambda: _tree(lse=BASE + MB)),
    (L.TC_E_ALIAS, "the cache", lambda: _tree(max_len=5000, work=BASE)),
    (L.TC_E_ALIAS, "an output", lambda: _tree(out=BASE + 4 * MB)),
    (L.TC_E_ALIAS, "an output", lambda: _tree(masks=BASE + 8 * MB)),
    (L.TC_E_ALIAS, "an output", lambda: _tree(lse=BASE + 16 * MB)),
    (L.TC_E_ALIAS, "an output", lambda: _tree(max_len=5000, work=BASE + 17 * MB)),
    (L.TC_E_ALIAS, "two outputs", lambda: _tree(lse=BASE + 8 * MB)),
    (L.TC_E_ALIAS, "two outputs", lambda: _tree(max_len=5000, work=BASE + 8 * MB)),
]
RESIZE = [
    (L.TC_E_NULL, "block_table", lambda: _resize(table=None)),
    (L.TC_E_RANK, "block_table", lambda: _resize(shape=(3, 4, 5))),
    (L.TC_E_NONINJECTIVE, "block_table", lambda: _resize(stride=(0, 1))),
    (L.TC_E_ARG, "negative", lambda: _resize(stride=(4, -1))),
    (L.TC_E_EXTENT, "page_size", lambda: _resize(page=0)),
    (L.TC_E_EXTENT, "page_size", lambda: _resize(page=1 << 31)),
    (L.TC_E_RANGE, "entries", lambda: _resize(shape=(1 << 16, 1 << 15), table=BASE + (1 << 40))),
    (L.TC_E_RANGE, "free_capacity", lambda: _resize(capacity=-1)),
    (L.TC_E_RANGE, "free_capacity", lambda: _resize(capacity=1 << 31)),
    (L.TC_E_RANGE, "tokens", lambda: _resize(tokens=-1)),
    (L.TC_E_RANGE, "tokens", lambda: _resize(tokens=1 << 31)),
    (L.TC_E_NULL, "seq_lens", lambda: _resize(lens=None)),
    (L.TC_E_NULL, "change", lambda: _resize(change=None)),
    (L.TC_E_NULL, "free_pages", lambda: _resize(free=None)),
    (L.TC_E_NULL, "free_count", lambda: _resize(count=None)),
    (L.TC_E_NULL, "lens_out", lambda: _resize(lens_out=None)),
    (L.TC_E_NULL, "count_out", lambda: _resize(count_out=None)),
    (L.TC_E_NULL, "need token_starts", lambda: _resize(starts=None, slots=BASE + 8 * MB, tokens=4)),
    (L.TC_E_NULL, "need token_starts", lambda: _resize(starts=None, positions=BASE + 8 * MB, tokens=4)),
    (L.TC_E_ALIGN, "slots", lambda: _resize(slots=BASE + 8 * MB + 4, tokens=4)),
    (L.TC_E_ALIGN, "seq_lens", lambda: _resize(lens=BASE + MB + 2)),
    (L.TC_E_ALIAS, "change", lambda: _resize(lens_out=BASE + 2 * MB)),
    (L.TC_E_ALIAS, "seq_lens", lambda: _resize(lens_out=BASE + MB + 4)),
    (L.TC_E_ALIAS, "seq_lens", lambda: _resize(missing=BASE + MB)),
    (L.TC_E_ALIAS, "free_count", lambda: _resize(starts=BASE + 4 * MB)),
    (L.TC_E_ALIAS, "two outputs", lambda: _resize(free=BASE)),
    (L.TC_E_ALIAS, "two outputs", lambda: _resize(slots=BASE + 7 * MB, tokens=4)),
    (L.TC_E_ALIAS, "two outputs", lambda: _resize(slots=BASE + 8 * MB, positions=BASE + 8 * MB + 16, tokens=4)),
    (L.TC_E_ALIAS, "two outputs", lambda: _resize(missing=BASE + 6 * MB)),
]


@pytest.mark.parametrize("want, word, call", PROMPT + TREE + RESIZE)
def test_refusals(want, word, call):
    rc = call()
    assert rc == want, (L.STATUS_NAMES.get(rc, rc), L.tc_last_error())
    assert word in L.tc_last_error()


@pytest.mark.parametrize("args, want", [((1, 1, 3, 2, 64, 100), L.TC_E_EXTENT), ((1, 1, 2, 2, 65, 100), L.TC_E_EXTENT),
                                        ((1, -1, 2, 2, 64, 100), L.TC_E_EXTENT), ((1, 1, 2, 2, 64, -1), L.TC_E_RANGE),
                                        ((1, 1 << 30, 2, 2, 64, 10), L.TC_E_RANGE), ((1, 1, 2, 0, 64, 10), L.TC_E_EXTENT)])
def test_workspace_refusals(args, want):
    assert L.load_library().tc_paged_tree_attention_workspace(*args) == want


def test_a_workspace_suffices_for_smaller_calls():
    """What sizes need, no smaller batch, tokens or max_len needs more of: what a call refuses as too small says so."""
    lib = L.load_library()
    size = lib.tc_paged_tree_attention_workspace
    for heads, group, dim in ((8, 4, 128), (1, 1, 16), (2, 8, 256), (16, 1, 64)):
        for batch, tokens, most in ((32, 512, 4096), (1, 64, 131072), (64, 64, 600), (3, 2000, 9000)):
            held = size(batch, tokens, heads * group, heads, dim, most)
            assert held >= 0
            for b in {1, max(1, batch // 2), max(1, batch - 1), batch}:
                for t in {0, 1, 7, tokens // 3, tokens}:
                    for m in {0, 512, 513, most // 2, most}:
                        assert size(b, t, heads * group, heads, dim, m) <= held
                        # the call itself needs no more: with one byte less than it would need it is refused for that
                        c = _cache(shape=(4096, 16, heads, dim), v=BASE + (1 << 33))
                        rc = _tree(c, q=BASE + (1 << 34), q_shape=(t, heads * group, dim), out=BASE + (1 << 35), table=(b, 4),
                                   max_len=m, work=BASE + (1 << 36) + 8, work_bytes=held, lens=BASE + (1 << 37), starts=BASE + (1 << 38))
                        assert rc in (L.TC_E_ALIGN, L.TC_E_ALIAS) or t == 0, (rc, L.tc_last_error())


def test_the_binding_refuses_on_the_host():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        L.tc_prompt_attention(t(3, 2, 64), t(3, 1, 64), t(3, 1, 64), i(2))
    with pytest.raises(ValueError, match="q is"):
        L.tc_prompt_attention(t(3, 2, 64), t(3, 1, 64, dt=torch.float16), t(3, 1, 64), i(2))
    with pytest.raises(ValueError, match="token_starts"):
        L.tc_prompt_attention(t(3, 2, 64), t(3, 1, 64), t(3, 1, 64), i(2).long())
    with pytest.raises(ValueError, match="key_starts"):
        L.tc_prompt_attention(t(3, 2, 64), t(3, 1, 64), t(3, 1, 64), i(2), key_starts=i(3))
    with pytest.raises(ValueError, match="q must"):
        L.tc_prompt_attention(t(3, 128), t(3, 1, 64), t(3, 1, 64), i(2))
    with pytest.raises(ValueError, match="lse"):
        L.tc_prompt_attention(t(3, 2, 64), t(3, 1, 64), t(3, 1, 64), i(2), lse=t(3, 2))
    cache = L.PagedCache(t(4, 16, 1, 64), t(4, 16, 1, 64))
    with pytest.raises(ValueError, match="on a GPU"):
        L.tc_paged_tree_attention(t(3, 2, 64), cache, i(1, 4), i(1), i(2))
    with pytest.raises(ValueError, match="masks"):
        L.tc_paged_tree_attention(t(3, 2, 64), cache, i(1, 4), i(1), i(2), masks=i(3))
    with pytest.raises(ValueError, match="masks"):
        L.tc_paged_tree_attention(t(3, 2, 64), cache, i(1, 4), i(1), i(2), masks=i(2).long())
    with pytest.raises(ValueError, match="token_starts"):
        L.tc_paged_tree_attention(t(3, 2, 64), cache, i(1, 4), i(1), i(3))
    with pytest.raises(ValueError, match="block_table"):
        L.tc_paged_tree_attention(t(3, 2, 64), cache, i(4), i(1), i(2))
    with pytest.raises(ValueError, match="on a GPU"):
        L.tc_paged_resize(i(2, 4), i(2), i(2), i(9), i(1), 16)
    for bad in (dict(change=i(3)), dict(free_count=i(2)), dict(seq_lens=i(2).long()), dict(slots=i(4), token_starts=i(3)),
                dict(positions=i(4).long(), token_starts=i(3)), dict(token_starts=i(2)), dict(missing=i(2)),
                dict(slots=i(4).long(), positions=i(5), token_starts=i(3))):
        args = dict(block_table=i(2, 4), seq_lens=i(2), change=i(2), free_pages=i(9), free_count=i(1), page_size=16)
        args.update(bad)
        with pytest.raises(ValueError):
            L.tc_paged_resize(**args)
    with pytest.raises(ValueError, match="block_table"):
        L.tc_paged_resize(i(2), i(2), i(2), i(9), i(1), 16)
    assert ctypes.sizeof(L.TcPagedCache) > 0


@pytest.mark.parametrize("args, want", [((1, 1, 1, 3, 2, 64), L.TC_E_EXTENT), ((1, 1, -1, 2, 2, 64), L.TC_E_RANGE), ((1, 1, 1, 2, 2, 65), L.TC_E_EXTENT),
                                        ((-1, 1, 1, 2, 2, 64), L.TC_E_EXTENT), ((0, 5, 5, 2, 2, 64), 0), ((1, 0, 5, 2, 2, 64), 0),
                                        ((1, 1, 1536, 2, 2, 64), 0), ((1, 1 << 20, 1 << 20, 8, 8, 64), 0)])
def test_prompt_workspace_sizes(args, want):
    assert L.load_library().tc_prompt_attention_workspace(*args) == want


def test_tree_workspace_suffices_for_smaller_calls():
    """What is asked at the largest sizes covers every call of fewer sequences, tokens and rows."""
    import random
    rng = random.Random(3)
    size = L.load_library().tc_paged_tree_attention_workspace
    for _ in range(3000):
        heads, group, dim = rng.choice([1, 2, 8, 40]), rng.choice([1, 4, 7, 16]), 16 * rng.randint(1, 16)
        batch, tokens, longest = rng.randint(1, 300), rng.randint(1, 3000), rng.choice([100, 513, 5000, 100000])
        most = size(batch, tokens, heads * group, heads, dim, longest)
        for _ in range(4):
            assert size(rng.randint(1, batch), rng.randint(1, tokens), heads * group, heads, dim, rng.randint(1, longest)) <= most
