"""Attention of several query rows at the ends of its ranges: values near the end of fp32's."""

import pytest
import torch

import layout_permuting_copy_amd as L
import paged_ref as P
import rows_ref as R
from gpu_util import say
from test_gpu_rows import _prompt, _random_masks, _tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load_library()
    yield
    torch.cuda.synchronize()


def _rising(rows, heads, dim, tokens, q_heads, a_step, gen):
    """Queries of ones in element 0, keys that rise by one in `a_step` rows there, values of about 3e38 / (2 a_step): the sums
    of exp(x - max x) |v| are half of fp32's range at most, however slowly the maximum grows."""
    q, k = torch.zeros(tokens, q_heads, dim, dtype=torch.bfloat16), torch.zeros(rows, heads, dim, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    k[:, :, 0] = (torch.arange(rows) / a_step)[:, None].to(torch.bfloat16)
    v = (torch.rand(rows, heads, dim, generator=gen) + 1) * torch.where(torch.rand(rows, heads, dim, generator=gen) < 0.2, -1.0, 1.0)
    return q, k, v * (3e38 / (4 * a_step))


@pytest.mark.parametrize("dim", [32, 80, 128, 192, 256])
@pytest.mark.parametrize("tokens, rows", [(300, 300), (7, 4000)])
def test_prompt_values_near_the_end_of_the_range(dim, tokens, rows):
    gen = torch.Generator().manual_seed(dim)
    q, k, v = _rising(rows, 1, dim, tokens, 2, rows // 15, gen)
    out, _, ref = _prompt(q, k, v.to(torch.bfloat16), [tokens], [rows], scale=1.0)
    assert bool(out.isfinite().all()) and float(ref[0].abs().max()) > 1e36 / rows


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [32, 128, 256])
@pytest.mark.parametrize("tokens, rows", [(5, 300), (5, 4000), (40, 300), (300, 1200)])
def test_tree_values_near_the_end_of_the_range(kind, dim, tokens, rows):
    """In tiles of each size, whole and in parts; 8-bit rows by their scales."""
    gen = torch.Generator().manual_seed(dim + rows)
    table, pages = P.table_for([rows], 16, gen)
    pool = P.Pool(kind, pages, 16, 1, dim, "rows", gen)
    q, k, v = _rising(rows, 1, dim, tokens, 2, rows // 15, gen)
    at, row = table[0][torch.arange(rows) // 16].long(), torch.arange(rows) % 16
    if kind == "e4m3":
        codes = lambda x: P.bits(x.to(torch.float8_e4m3fn))
        P.bits(pool.k)[at, row] = codes(k.float().sign())
        pool.ks[at, row] = k.float().amax(-1)
        P.bits(pool.v)[at, row] = codes(v / v.abs().amax(-1, keepdim=True))
        pool.vs[at, row] = v.abs().amax(-1)
    else:
        pool.k[at, row], pool.v[at, row] = k, v.to(torch.bfloat16)
    say(f"[gpu] {tokens} tokens over {rows} rows of {dim}")
    for words in (None, _random_masks(gen, tokens, "tree")):
        out, _, ref = _tree(q, pool, table, [rows], [tokens], 16, words, scale=1.0, max_len=rows)
        assert bool(out.isfinite().all()) and float(ref[0].abs().max()) > 1e36 / rows
