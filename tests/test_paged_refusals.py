"""The paged cache entry points refuse what they cannot do, before anything is launched: host only, the device
addresses are never dereferenced."""

import ctypes

import pytest

import layout_permuting_copy_amd as L

PAGES, PAGE, HEADS, DIM = 8, 16, 2, 64
BASE = 0x10000000


def _lay(shape, stride=None, offset=0):
    return L.make_layout(shape, stride, offset)


def _cache(dtype=L.TC_BF16, k=BASE, v=BASE + (1 << 20), shape=(PAGES, PAGE, HEADS, DIM), k_stride=None, v_stride=None, ks=None, vs=None,
           offset=0):
    c = L.TcPagedCache()
    c.dtype, c.k, c.v, c.k_scale, c.v_scale = dtype, k, v, ks, vs
    c.k_layout, c.v_layout = _lay(shape, k_stride, offset), _lay(shape, v_stride)
    c.k_scale_layout = c.v_scale_layout = _lay(shape[:3])
    return c


def _ref(x):
    return None if x is None else ctypes.addressof(x)


def _append(cache=None, dtype=L.TC_BF16, new=(3, HEADS, DIM), k=BASE + (4 << 20), v=BASE + (5 << 20), table=(3, 4), starts=None,
            lens=BASE + (7 << 20), w=None, w_shape=(3, HEADS, 64), k_stride=None):
    cache = _cache() if cache is None else cache
    kl, vl, tl, wl = _lay(new, k_stride), _lay(new), _lay(table), _lay(w_shape)
    return L.load_library().tc_paged_append(_ref(cache), k, _ref(kl), v, _ref(vl), dtype, BASE + (6 << 20), _ref(tl), lens, starts,
                                            w, _ref(wl), None)


def _attend(cache=None, dtype=L.TC_BF16, q=BASE + (4 << 20), q_shape=(3, 4, DIM), out=BASE + (5 << 20), out_shape=None, table=(3, 4),
            max_len=64, scale=1.0, lse=None, lse_shape=(3, 4), w=None, wo=None, w_shape=(3, HEADS, 64), work=BASE + (256 << 20),
            work_bytes=1 << 26, out_stride=None, lens=BASE + (7 << 20)):
    cache = _cache() if cache is None else cache
    ql, ol, tl, ll, wl = _lay(q_shape), _lay(out_shape or q_shape, out_stride), _lay(table), _lay(lse_shape), _lay(w_shape)
    return L.load_library().tc_paged_attention(_ref(cache), q, _ref(ql), out, _ref(ol), dtype, BASE + (6 << 20), _ref(tl), lens, max_len,
                                               scale, lse, _ref(ll), w, _ref(wl), wo, _ref(wl), work, work_bytes, None)


def _evict(src=None, dst=None, table=(3, 4), dst_table=(3, 4), budget=32, recent=8, w_shape=(3, HEADS, 64), kept=BASE + (20 << 20),
           kept_shape=(3, HEADS, 32), lens_out=BASE + (21 << 20), wo=None, wo_shape=(3, HEADS, 32), max_len=64, lens=BASE + (7 << 20),
           w=BASE + (22 << 20)):
    src = _cache() if src is None else src
    dst = _cache(k=BASE + (30 << 20), v=BASE + (31 << 20)) if dst is None else dst
    tl, wl, dl, kl, wol = _lay(table), _lay(w_shape), _lay(dst_table), _lay(kept_shape), _lay(wo_shape)
    return L.load_library().tc_paged_evict(_ref(src), BASE + (6 << 20), _ref(tl), lens, max_len, w, _ref(wl), _ref(dst),
                                           BASE + (23 << 20), _ref(dl), budget, recent, lens_out, kept, _ref(kl), wo, _ref(wol), None)


BIG = 1 << 59


@pytest.mark.parametrize("want, word, call", [
    (L.TC_E_NULL, "null cache", lambda: L.load_library().tc_paged_append(None, 1, None, 1, None, L.TC_BF16, 1, None, 1, None, None, None, None)),
    (L.TC_E_DTYPE, "dtype", lambda: _append(_cache(dtype=L.TC_F32))),
    (L.TC_E_DTYPE, "dtype", lambda: _append(dtype=L.TC_F32)),
    (L.TC_E_DTYPE, "differ in type", lambda: _append(dtype=L.TC_F16)),
    (L.TC_E_EXTENT, "head_dim", lambda: _append(_cache(shape=(PAGES, PAGE, HEADS, 72)), new=(3, HEADS, 72))),
    (L.TC_E_EXTENT, "head_dim", lambda: _append(_cache(shape=(PAGES, PAGE, HEADS, 272)), new=(3, HEADS, 272))),
    (L.TC_E_EXTENT, "page_size", lambda: _append(_cache(shape=(PAGES, 0, HEADS, DIM)))),
    (L.TC_E_EXTENT, "shape", lambda: _append(new=(3, HEADS + 1, DIM))),
    (L.TC_E_EXTENT, "one token", lambda: _append(new=(4, HEADS, DIM))),
    (L.TC_E_ALIGN, "16-byte", lambda: _append(_cache(k=BASE + 8))),
    (L.TC_E_ALIGN, "16-byte", lambda: _append(_cache(offset=4))),
    (L.TC_E_ALIGN, "16-byte", lambda: _append(_cache(k_stride=(PAGE * HEADS * 68, HEADS * 68, 68, 1)))),
    (L.TC_E_ALIGN, "aligned", lambda: _append(k=BASE + (4 << 20) + 1)),
    (L.TC_E_ARG, "innermost", lambda: _append(_cache(k_stride=(PAGE * HEADS * DIM, HEADS * DIM, 1, HEADS)))),
    (L.TC_E_ARG, "innermost", lambda: _append(k_stride=(2 * HEADS * DIM, 2 * DIM, 2))),
    (L.TC_E_ARG, "negative", lambda: _append(k_stride=(-HEADS * DIM, DIM, 1))),
    (L.TC_E_NONINJECTIVE, "two indices", lambda: _append(_cache(k_stride=(0, HEADS * DIM, DIM, 1)))),
    (L.TC_E_NONINJECTIVE, "two indices", lambda: _append(_cache(k_stride=(HEADS * DIM, HEADS * DIM, DIM, 1)))),
    (L.TC_E_NONINJECTIVE, "weights", lambda: _append_w0()),
    (L.TC_E_ALIAS, "keys and values", lambda: _append(_cache(v=BASE + 128))),
    (L.TC_E_ALIAS, "overlaps", lambda: _append(k=BASE + 64)),
    (L.TC_E_ALIAS, "overlaps", lambda: _append(lens=BASE + 64)),
    (L.TC_E_RANGE, "2^58", lambda: _append(_cache(k_stride=(BIG, HEADS * DIM, DIM, 1)))),
    (L.TC_E_RANGE, "2^58", lambda: _append(_cache(offset=BIG))),
    (L.TC_E_NULL, "k_scale", lambda: _append(_cache(dtype=L.TC_E4M3))),
    (L.TC_E_ARG, "scales", lambda: _append(_cache(ks=BASE + (25 << 20), vs=BASE + (26 << 20)))),
    (L.TC_E_ALIAS, "scales", lambda: _append(_cache(dtype=L.TC_E4M3, ks=BASE + (25 << 20), vs=BASE + (25 << 20)))),
    (L.TC_E_EXTENT, "weights", lambda: _append(w=BASE + (24 << 20), w_shape=(3, HEADS + 1, 64))),
    (L.TC_E_EXTENT, "multiple", lambda: _attend(q_shape=(3, 3, DIM))),
    (L.TC_E_EXTENT, "head_dim", lambda: _attend(q_shape=(3, 4, 80))),
    (L.TC_E_EXTENT, "q and out", lambda: _attend(out_shape=(3, 4, 80))),
    (L.TC_E_EXTENT, "batch", lambda: _attend(table=(2, 4))),
    (L.TC_E_EXTENT, "lse", lambda: _attend(lse=BASE + (8 << 20), lse_shape=(4, 3))),
    (L.TC_E_EXTENT, "weights", lambda: _attend(w=BASE + (24 << 20), wo=BASE + (24 << 20), w_shape=(3, HEADS, 63))),
    (L.TC_E_NULL, "together", lambda: _attend(wo=BASE + (24 << 20))),
    (L.TC_E_ARG, "scale", lambda: _attend(scale=float("nan"))),
    (L.TC_E_RANGE, "max_len", lambda: _attend(max_len=1 << 31)),
    (L.TC_E_RANGE, "max_len", lambda: _attend(max_len=-1)),
    (L.TC_E_ARG, "workspace", lambda: _attend(table=(3, 400), max_len=6000, work_bytes=64)),
    (L.TC_E_NULL, "workspace", lambda: _attend(table=(3, 400), max_len=6000, work=None)),
    (L.TC_E_ALIGN, "workspace", lambda: _attend(table=(3, 400), max_len=6000, work=BASE + (256 << 20) + 8)),
    (L.TC_E_ALIAS, "input", lambda: _attend(out=BASE + (4 << 20))),
    (L.TC_E_ALIAS, "cache", lambda: _attend(out=BASE + (1 << 20))),
    (L.TC_E_ALIAS, "overlap", lambda: _attend(w=BASE + (24 << 20), wo=BASE + (24 << 20) + 4)),
    (L.TC_E_ALIAS, "outputs", lambda: _attend(table=(3, 400), max_len=6000, work=BASE + (5 << 20))),
    (L.TC_E_NONINJECTIVE, "out", lambda: _attend(out_stride=(0, DIM, 1))),
    (L.TC_E_NULL, "seq_lens", lambda: _attend(lens=None)),
    (L.TC_E_ARG, "recent", lambda: _evict(recent=33)),
    (L.TC_E_ARG, "recent", lambda: _evict(recent=-1)),
    (L.TC_E_ARG, "budget", lambda: _evict(budget=0, recent=0)),
    (L.TC_E_EXTENT, "dst_table", lambda: _evict(dst_table=(3, 1))),
    (L.TC_E_EXTENT, "kept", lambda: _evict(kept_shape=(3, HEADS, 31))),
    (L.TC_E_EXTENT, "weights_out", lambda: _evict(wo=BASE + (24 << 20), wo_shape=(3, HEADS, 31))),
    (L.TC_E_EXTENT, "weights", lambda: _evict(w_shape=(3, HEADS, 63))),
    (L.TC_E_EXTENT, "tables", lambda: _evict(dst_table=(2, 4))),
    (L.TC_E_EXTENT, "head", lambda: _evict(dst=_cache(k=BASE + (30 << 20), v=BASE + (31 << 20), shape=(PAGES, PAGE, HEADS + 1, DIM)))),
    (L.TC_E_DTYPE, "type", lambda: _evict(dst=_cache(dtype=L.TC_F16, k=BASE + (30 << 20), v=BASE + (31 << 20)))),
    (L.TC_E_ALIAS, "same pool", lambda: _evict(dst=_cache(k=BASE + 4096, v=BASE + (31 << 20)))),
    (L.TC_E_ALIAS, "input", lambda: _evict(lens_out=BASE + (7 << 20))),
    (L.TC_E_ALIAS, "input", lambda: _evict(wo=BASE + (22 << 20))),
    (L.TC_E_NULL, "kept", lambda: _evict(kept=None)),
    (L.TC_E_RANGE, "one launch", lambda: _append(new=(1 << 28, HEADS, DIM), k_stride=(0, DIM, 1), starts=BASE + (8 << 20))),
    (L.TC_E_RANGE, "one launch", lambda: _attend(q_shape=(1 << 23, 4, DIM), q=1 << 40, out=1 << 42, lens=1 << 44, table=(1 << 23, 4))),
    (L.TC_E_RANGE, "one launch", lambda: _attend(_cache(shape=(PAGES, PAGE, 1, DIM)), q_shape=(1 << 12, 1, DIM), q=1 << 40, out=1 << 42,
                                                 lens=1 << 44, table=(1 << 12, 1 << 16), max_len=1 << 20, w=1 << 50, wo=1 << 50,
                                                 w_shape=(1 << 12, 1, 1 << 20), work=1 << 52, work_bytes=1 << 40)),
    (L.TC_E_RANGE, "one launch", lambda: _evict(table=(1 << 23, 4), dst_table=(1 << 23, 4), kept=1 << 40, lens_out=1 << 42,
                                                kept_shape=(1 << 23, HEADS, 32), w=1 << 44, w_shape=(1 << 23, HEADS, 64), lens=1 << 46,
                                                dst=_cache(k=1 << 47, v=1 << 48))),
])
def test_refusals(want, word, call):
    assert call() == want, L.tc_last_error()
    assert word in L.tc_last_error()


def _append_w0():
    cache, new, table = _cache(), _lay((3, HEADS, DIM)), _lay((3, 4))
    w = _lay((3, HEADS, 64), (0, 64, 1))
    return L.load_library().tc_paged_append(_ref(cache), BASE + (4 << 20), _ref(new), BASE + (5 << 20), _ref(new), L.TC_BF16,
                                            BASE + (6 << 20), _ref(table), BASE + (7 << 20), None, BASE + (24 << 20), _ref(w), None)


def test_workspace_sizes():
    lib = L.load_library()
    size = lib.tc_paged_attention_workspace
    assert size(4, 32, 8, 128, 0, 0) == 0 and size(0, 32, 8, 128, 4096, 1) == 0
    assert size(1, 32, 8, 128, 64, 0) == 0  # one split: the outputs are written at once
    long = size(1, 32, 8, 128, 131072, 0)
    assert 0 < long < 2 * 131072 * 8 * 128 * 2 // 8  # well under the cache that it stands beside
    assert size(1, 32, 8, 128, 131072, 1) >= long + 32 * 131072 * 4
    assert size(1, 33, 8, 128, 64, 0) == L.TC_E_EXTENT and "multiple" in L.tc_last_error()
    assert size(1, 32, 8, 129, 64, 0) == L.TC_E_EXTENT
    assert size(1 << 30, 1 << 30, 8, 128, 64, 0) == L.TC_E_RANGE


def test_interlaced_pools_are_accepted():
    """Keys and values as halves of one allocation, a page or a row or a head apart, are no overlap: the call gets
    past the cache's checks to the next argument's."""
    n = PAGE * HEADS * DIM
    for stride, gap in (((2 * n, HEADS * DIM, DIM, 1), n), ((2 * n, 2 * HEADS * DIM, DIM, 1), HEADS * DIM),
                        ((2 * n, 2 * HEADS * DIM, 2 * DIM, 1), DIM)):
        c = _cache(k_stride=stride, v_stride=stride, v=BASE + 2 * gap)
        assert _append(c, new=(3, HEADS, 80)) == L.TC_E_EXTENT and "of the cache" in L.tc_last_error()
        c = _cache(k_stride=stride, v_stride=stride, v=BASE + 2 * gap - 16)
        assert _append(c) == L.TC_E_ALIAS


def test_tensor_checks():
    """What the tensors themselves get wrong is refused by the binding."""
    import torch
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    k = z(PAGES, PAGE, HEADS, DIM)
    cache = L.PagedCache(k, k.clone())
    assert (cache.pages, cache.page_size, cache.heads, cache.head_dim) == (PAGES, PAGE, HEADS, DIM)
    with pytest.raises(ValueError):
        L.PagedCache(k, k.half())
    with pytest.raises(ValueError):
        L.PagedCache(k, k.clone(), z(PAGES, PAGE, HEADS, dt=torch.float32), None)
    with pytest.raises(ValueError):
        L.PagedCache(k.float(), k.float())
    with pytest.raises(ValueError):
        L.PagedCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn))
    table, lens = z(3, 4, dt=torch.int32), z(3, dt=torch.int32)
    q = z(3, 4, DIM)
    for call in (lambda: L.tc_paged_attention(q, cache, table, lens),  # not on a GPU
                 lambda: L.tc_paged_attention(q, cache, table.long(), lens),
                 lambda: L.tc_paged_attention(q, cache, table, lens[:2]),
                 lambda: L.tc_paged_attention(q, cache, table, z(6, dt=torch.int32)[::2]),
                 lambda: L.tc_paged_attention(q, cache, table, lens, weights=z(3, HEADS, 64)),
                 lambda: L.tc_paged_attention(q, cache, table, lens, weights_out=z(3, HEADS, 64, dt=torch.float32)),
                 lambda: L.tc_paged_attention(q.float(), cache, table, lens),
                 lambda: L.tc_paged_append(cache, z(3, HEADS, DIM), z(3, HEADS, DIM, dt=torch.float16), table, lens),
                 lambda: L.tc_paged_append(cache, z(3, HEADS, DIM), z(3, HEADS, DIM), table, lens, token_starts=lens),
                 lambda: L.tc_paged_evict(cache, table, lens, z(3, HEADS, 64), cache, table, 8)):
        with pytest.raises(ValueError):
            call()


def test_8bit_floats_copy_as_bytes():
    p = L.tc_plan(((64, 128), (128, 1)), ((64, 128), (1, 64)), L.TC_E4M3)
    q = L.tc_plan(((64, 128), (128, 1)), ((64, 128), (1, 64)), L.TC_I8)
    assert p == q and p["elem_bytes"] == 1
