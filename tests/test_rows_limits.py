"""Grids of the attention of several rows at the limit of a launch: host only, the device addresses are never
dereferenced."""

import pytest
import torch

import layout_permuting_copy_amd as L
from test_paged_refusals import PAGE, PAGES, _cache
from test_rows_refusals import _prompt, _tree

AT = 1 << 40


def _sequences(workgroups, tile):
    """So many one-token sequences make fewer workgroups, one more does not: a workgroup each, and one for each tile of tokens."""
    n = workgroups * tile // (tile + 1) - 2
    while n + 1 + (n + 1) // tile < workgroups:
        n += 1
    return n


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that passes the checks would be launched on made-up addresses")
@pytest.mark.parametrize("dim, lanes, prompt_tile, tree_tile", [(64, 256, 64, 64), (128, 256, 64, 64), (144, 512, 128, 128), (256, 512, 128, 128)])
def test_attention_is_refused_only_past_its_own_grid(dim, lanes, prompt_tile, tree_tile):
    """Workgroups have eight waves for heads above 128 elements but over 8-bit rows: calls of just under 2^32 lanes go on to the launch (which
    finds no GPU here), calls of 2^32 are refused."""
    most = _sequences(2 ** 32 // lanes, prompt_tile)
    for tokens, want in ((most, L.TC_E_HIP), (most + 1, L.TC_E_RANGE)):
        rc = _prompt(q_shape=(tokens, 1, dim), k_shape=(tokens, 1, dim), q=AT, k=2 * AT, v=3 * AT, out=4 * AT, starts=5 * AT, batch=tokens)
        assert rc == want, (tokens, rc, L.tc_last_error())
    for dtype, kind in ((L.TC_BF16, L.TC_BF16), (L.TC_F16, L.TC_F16), (L.TC_F16, L.TC_E4M3), (L.TC_BF16, L.TC_E4M3)):
        scales = dict(ks=9 * AT, vs=10 * AT) if kind == L.TC_E4M3 else {}
        cache = _cache(kind, shape=(PAGES, PAGE, 1, dim), k=6 * AT, v=7 * AT, **scales)
        most = _sequences(2 ** 32 // (256 if scales else lanes), tree_tile)
        for tokens, want in ((most, L.TC_E_HIP), (most + 1, L.TC_E_RANGE)):
            rc = _tree(cache, dtype=dtype, q_shape=(tokens, 1, dim), q=AT, out=4 * AT, starts=5 * AT, lens=8 * AT, table=(tokens, 1), max_len=64)
            assert rc == want, (tokens, rc, L.tc_last_error())
