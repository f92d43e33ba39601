"""Attention of several query rows in tiles that only calls of many heads or rows take, and how many bits weights keep there,
against the definitions in 64 bits on the host."""

import pytest
import torch

import layout_permuting_copy_amd as L
import paged_ref as P
import rows_ref as R
from gpu_util import say
from test_gpu_rows import LARGE, TREES, _i32, _prompt, _prompt_ref, _qkv, _random_masks, _tree, _tree_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load_library()
    yield
    torch.cuda.synchronize()


# key heads, heads a group, head_dim, tokens, keys: at least 1024 tiles of 128 rows, and fewer than 2048 rows a sequence
MANY_TILES = [(128, 1, 32, [300, 1, 0, 129, 260], [300, 40, 7, 129, 400]), (176, 1, 64, [513, 70], [513, 200]), (96, 2, 80, [128, 400, 3], None),
              (104, 1, 96, [640, 257, 20], [641, 100, 20]), (104, 3, 112, [300, 41], [350, 41]), (144, 1, 128, [700, 129], None)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", MANY_TILES, ids=lambda s: "x".join(map(str, s[:3])))
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_of_many_heads(kind, shape, causal):
    """Tiles of 128 rows, ragged and past the keys' end; all heads are copies of two, and equal to them."""
    heads, group, dim, n, m = shape
    gen = torch.Generator().manual_seed(dim)
    m = n if m is None else m
    q, k, v = _qkv(gen, P.DT[kind], sum(n) + 3, sum(m) + 3, 2, group, dim)
    k[sum(m):], v[sum(m):] = torch.nan, torch.inf
    kv = torch.arange(heads) % 2
    qs = (kv[:, None] * group + torch.arange(group)).flatten()
    out, lse = torch.full((sum(n) + 3, heads * group, dim), 7.0, dtype=q.dtype, device="cuda"), torch.full((sum(n) + 3, heads * group), 7.0, device="cuda")
    say(f"[gpu] {n} tokens over {m} keys, {heads} x {group} heads of {dim}")
    L.tc_prompt_attention(q.cuda()[:, qs], k.cuda()[:, kv], v.cuda()[:, kv], _i32(R.starts_of(n)), key_starts=_i32(R.starts_of(m)),
                          causal=causal, out=out, lse=lse)
    ref = _prompt_ref(q, k, v, n, m, causal)
    total, two = sum(n), 2 * group
    R.close(out[:total, :two], ref[0], ref[2], "out", q.dtype)
    R.close(lse[:total, :two], ref[1], ref[3], "lse")
    for x in (out, lse):
        assert torch.equal(x, x[:, :two].repeat(1, heads // 2, *[1] * (x.dim() - 2)))
        assert bool((x[total:] == 7.0).all())


SMALL = [  # heads, group, dim, page, major, lens, tokens: at most 32 query rows a sequence on average
    (2, 4, 64, 16, "heads", [400, 7, 0, 140], [8, 7, 0, 1]), (1, 3, 80, 7, "rows", [65, 929, 64], [5, 20, 7]), (1, 8, 128, 16, "pairs", [1000, 513], [2, 6]),
    (2, 1, 32, 4, "rows", [3000], [30]), (4, 2, 112, 64, "heads", [200, 64, 65], [16, 1, 20]), (3, 2, 48, 24, "rows", [130], [16])]


def _case(shape, cache, dtype):
    heads, group, dim, page, major, lens, n = shape
    gen = torch.Generator().manual_seed(dim + page)
    table, pages = P.table_for(lens, page, gen, spare=1)
    pool = P.Pool(cache, pages, page, heads, dim, major, gen)
    q = torch.randn(sum(n), heads * group, dim, generator=gen).to(dtype)
    out = L.tc_paged_tree_attention(q.cuda(), pool.on_gpu(), table.cuda(), _i32(lens), _i32(R.starts_of(n)))
    return q, pool, table, out


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SMALL, ids=lambda s: "x".join(map(str, s[:4])))
def test_bf16_in_tiles_of_64_rows_keeps_its_bits(shape, cache):
    """Weights there are the sum of two bf16 values, off by the square of half a bf16 step (2^-8)."""
    _, _, _, page, _, lens, n = shape
    q, pool, table, out = _case(shape, cache, torch.bfloat16)
    ref = _tree_ref(q, pool, table, lens, n, page, None, part=2.0 ** -16)
    R.close(out, ref[0], ref[2], "out", torch.bfloat16)


@pytest.mark.parametrize("shape", SMALL + TREES[:5] + LARGE, ids=lambda s: "x".join(map(str, s[:4])))
def test_fp16_trees_lose_only_what_subnormal_weights_do(shape):
    """Weights below 2^-21 of a row's greatest are subnormal fp16 numbers, off by 2^-32 of it at most: by the row's own values."""
    _, _, _, page, _, lens, n = shape
    q, pool, table, out = _case(shape, "fp16", torch.float16)
    a = 0
    for b, (t, m) in enumerate(zip(n, lens)):
        k, v = (pool.rows(x, table[b], m, page)[0].to(torch.float16) for x in ("k", "v"))
        ref = R.sequence(q[a:a + t], k, v, R.before(t, m))
        R.close(out[a:a + t], ref[0], ref[2], f"out of sequence {b}", torch.float16)
        a += t


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("group", [33, 65, 300])
def test_groups_of_more_heads_than_a_tile_has_rows(kind, group):
    """One key head under many query heads: a token's rows begin anywhere in a tile and end in another."""
    gen = torch.Generator().manual_seed(group)
    dt, dim, lens, n = P.DT[kind] if kind != "e4m3" else torch.bfloat16, 64, [90, 0, 700], [3, 0, 5]
    if kind != "e4m3":
        _prompt(*_qkv(gen, dt, 12, 12, 1, group, dim), [4, 0, 1, 6])
    table, pages = P.table_for(lens, 16, gen)
    pool = P.Pool(kind, pages, 16, 1, dim, "rows", gen)
    q = torch.randn(sum(n) + 1, group, dim, generator=gen).to(dt)
    say(f"[gpu] {group} heads a group")
    _tree(q, pool, table, lens, n, 16)
    _tree(q, pool, table, lens, n, 16, [w for t in n for w in _random_masks(gen, t, "any")])
