"""Pools that share memory between pages, grids at the limit of a launch, and workspaces of smaller calls: host only, the
device addresses are never dereferenced."""

import pytest
import torch

import layout_permuting_copy_amd as L
from test_paged_refusals import BASE, DIM, HEADS, PAGE, PAGES, _append, _attend, _cache, _evict


def _named(shape, stride, base):
    """The elements that a layout names, by brute force."""
    out = [base]
    for n, s in zip(shape, stride):
        out = [x + i * s for x in out for i in range(n)]
    return out


def _interlaced(stride, gap, pages=4):
    """Keys and values of one layout, the values `gap` elements on: what the append's check of the cache says."""
    shape = (pages, PAGE, HEADS, DIM)
    c = _cache(shape=shape, k_stride=stride, v_stride=stride, v=BASE + 2 * gap)
    rc = _append(c, new=(3, HEADS, 80))  # a refusal of the next argument's, where the cache passes
    share = bool(set(_named(shape, stride, 0)) & set(_named(shape, stride, gap)))
    return rc, L.tc_last_error(), share


R = HEADS * DIM


@pytest.mark.parametrize("stride, gap", [
    (((PAGE - 1) * 2 * R + R, 2 * R, DIM, 1), R),   # a page's last value row is the next page's first key row
    ((PAGE * 2 * R - 2 * R + DIM, 2 * R, DIM, 1), R),
    ((PAGE * 2 * R, 2 * R, DIM, 1), R + DIM // 2),  # half a head further: the last head's end is the next row's beginning
    ((PAGE * 4 * R, 2 * R, DIM, 1), R + 16),
    ((PAGE * 2 * R - R, 2 * R, DIM, 1), PAGE * 2 * R),
    ((2 * PAGE * R, R, DIM, 1), PAGE * R - R),
])
def test_pools_that_share_rows_are_refused(stride, gap):
    rc, why, share = _interlaced(stride, gap)
    assert share
    assert rc in (L.TC_E_ALIAS, L.TC_E_NONINJECTIVE), (rc, why)


@pytest.mark.parametrize("stride, gap", [
    ((PAGE * 2 * R, 2 * R, DIM, 1), R), ((2 * PAGE * R, R, DIM, 1), PAGE * R), ((PAGE * 2 * R, 2 * R, 2 * DIM, 1), DIM),
    ((PAGE * 2 * R + 16, 2 * R, DIM, 1), R), ((PAGE * 3 * R, 3 * R, DIM, 1), 2 * R), ((PAGE * 3 * R, 3 * R, DIM, 1), R),
    ((PAGE * R, R, DIM, 1), 4 * PAGE * R),
    ((DIM, 8 * DIM * HEADS, 8 * DIM, 1), 4 * DIM),  # pages fastest
])
def test_pools_that_share_nothing_pass(stride, gap):
    rc, why, share = _interlaced(stride, gap)
    assert not share
    assert rc == L.TC_E_EXTENT and "of the cache" in why, (rc, why)


def test_scales_that_share_rows_are_refused():
    """The scales of keys and values in one allocation, a row's heads apart, with a page stride that lets a page's last
    value scales be the next page's first key scales."""
    for page, want in ((2 * PAGE * HEADS, L.TC_E_EXTENT), ((PAGE - 1) * 2 * HEADS + HEADS, L.TC_E_ALIAS)):
        c = _cache(dtype=L.TC_E4M3, ks=BASE + (25 << 20), vs=BASE + (25 << 20) + 4 * HEADS)
        c.k_scale_layout = c.v_scale_layout = L.make_layout((PAGES, PAGE, HEADS), (page, 2 * HEADS, 1))
        assert _append(c, new=(3, HEADS, 80)) == want, L.tc_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that passes the checks would be launched on made-up addresses")
@pytest.mark.parametrize("dtype, dim, rows_a_workgroup", [
    (L.TC_BF16, 16, 128), (L.TC_BF16, 64, 32), (L.TC_BF16, 80, 16), (L.TC_BF16, 128, 16), (L.TC_BF16, 256, 8),
    (L.TC_E4M3, 16, 256), (L.TC_E4M3, 128, 32), (L.TC_E4M3, 144, 16), (L.TC_E4M3, 256, 16)])
def test_eviction_is_refused_only_past_its_own_grid(dtype, dim, rows_a_workgroup):
    """The copy takes 256 lanes for 4096 bytes of rows of a power of two: calls of just under 2^32 lanes go on to the launch
    (which finds no GPU here), calls of 2^32 are refused."""
    batch = 2048
    chunks = 2 ** 32 // 256 // (batch * HEADS)  # workgroups a sequence and head that make 2^32 lanes
    for most, want in (((chunks - 1) * rows_a_workgroup, L.TC_E_HIP), ((chunks - 1) * rows_a_workgroup + 1, L.TC_E_RANGE),
                       (chunks * rows_a_workgroup, L.TC_E_RANGE)):
        shape, at = (PAGES, 1 << 20, HEADS, dim), 1 << 40
        scales = [None] * 4 if dtype == L.TC_BF16 else [(40 + i) * at for i in range(4)]
        src = _cache(dtype, 1 * at, 2 * at, shape, ks=scales[0], vs=scales[1])
        dst = _cache(dtype, 3 * at, 4 * at, shape, ks=scales[2], vs=scales[3])
        rc = _evict(src, dst, table=(batch, 1), dst_table=(batch, 1), budget=most, recent=0, max_len=most, w=5 * at,
                    w_shape=(batch, HEADS, most), kept=6 * at, kept_shape=(batch, HEADS, most), lens_out=7 * at, lens=8 * at)
        assert rc == want, (most, rc, L.tc_last_error())


@pytest.mark.parametrize("q_heads, heads, dim", [(32, 8, 128), (1, 1, 64), (40, 2, 96), (20, 1, 256), (48, 48, 64)])
@pytest.mark.parametrize("weights", [0, 1])
def test_a_workspace_suffices_for_smaller_calls(q_heads, heads, dim, weights):
    """The workspace of a batch and max_len is enough for every smaller one, as a serving loop or graphs of several batch
    sizes allocate it once; a call that is given it gets past the check of its size."""
    size = L.load_library().tc_paged_attention_workspace
    batches, lengths = (1, 2, 7, 8, 16, 31, 32, 33, 64, 255, 256, 257, 1000), (1, 128, 511, 512, 513, 1000, 1024, 1025, 2048, 20000)
    grid = [[size(b, q_heads, heads, dim, n, weights) for n in lengths] for b in batches]
    assert min(map(min, grid)) >= 0
    for row in grid:
        assert row == sorted(row), (row, lengths)
    for column in zip(*grid):
        assert list(column) == sorted(column), (column, batches)
    cache = _cache(shape=(PAGES, PAGE, heads, dim), k=1 << 40, v=1 << 41)
    at = 1 << 42
    for b in batches:
        for n in lengths:  # out overlaps q: refused, but later than a small workspace is
            rc = _attend(cache, q=at, out=at, q_shape=(b, q_heads, dim), table=(b, 4), max_len=n, work=1 << 43, work_bytes=grid[-1][-1],
                         lens=1 << 44, w=1 << 45 if weights else None, wo=1 << 45 if weights else None, w_shape=(b, heads, n))
            assert rc == L.TC_E_ALIAS, (b, n, L.tc_last_error())
            rc = _attend(cache, q=at, out=at, q_shape=(b, q_heads, dim), table=(b, 4), max_len=n, work=1 << 43,
                         work_bytes=size(b, q_heads, heads, dim, n, weights), lens=1 << 44, w=1 << 45 if weights else None,
                         wo=1 << 45 if weights else None, w_shape=(b, heads, n))
            assert rc == L.TC_E_ALIAS, (b, n, L.tc_last_error())
