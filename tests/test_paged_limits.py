"""Pools that share memory between pages, grids at the limit of a launch, and workspaces of smaller calls: host only, the
device addresses are never dereferenced."""

import pytest

import layout_permuting_copy_amd as L
from test_paged_refusals import BASE, DIM, HEADS, PAGE, PAGES, _append, _cache


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
