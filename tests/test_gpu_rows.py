"""Attention of whole prompts and of each sequence's last tokens over its cache on the GPU, against the definitions in
64 bits on the host."""

import math
import threading

import pytest
import torch

import layout_permuting_copy_amd as L
import paged_ref as P
import rows_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.load_library()
    yield
    torch.cuda.synchronize()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _i64(x):
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in x], dtype=torch.int64, device="cuda")


def _prompt_ref(q, k, v, n, m, causal, scale=None):
    """out, lse and their tolerances, rows of no sequence NaN."""
    parts, a, c = [], 0, 0
    for x, y in zip(n, m):
        seen = R.before(x, y) if causal else torch.ones(x, y, dtype=torch.bool)
        parts.append(R.sequence(q[a:a + x], k[c:c + y], v[c:c + y], seen, scale))
        a, c = a + x, c + y
    return [torch.cat(p) for p in zip(*parts)]


def _prompt(q, k, v, n, m=None, causal=True, scale=None, devices=None, stream=None):
    """The call, its padding checked to be left alone; returns (out, lse) and the reference."""
    same = m is None
    m = n if same else m
    qd, kd, vd = devices or (q.cuda(), k.cuda(), v.cuda())
    out, lse = torch.full_like(qd, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    got = L.tc_prompt_attention(qd, kd, vd, _i32(R.starts_of(n)), key_starts=None if same else _i32(R.starts_of(m)), causal=causal,
                                scale=scale, out=out, lse=lse, stream=stream)
    torch.cuda.synchronize()
    assert got is out
    ref = _prompt_ref(q, k, v, n, m, causal, scale)
    total = sum(n)
    R.close(out[:total], ref[0], ref[2], "out", q.dtype)
    R.close(lse[:total], ref[1], ref[3], "lse")
    assert bool((out[total:] == 7.0).all()) and bool((lse[total:] == 7.0).all())
    return out, lse, ref


def _qkv(gen, dt, tokens, rows, heads, group, dim, spread=2.5):
    return ((spread * torch.randn(tokens, heads * group, dim, generator=gen)).to(dt), torch.randn(rows, heads, dim, generator=gen).to(dt),
            torch.randn(rows, heads, dim, generator=gen).to(dt))


SHAPES = [(1, 1, 16, [1]), (2, 4, 64, [0, 31, 33, 1, 129]), (1, 3, 80, [65, 0, 64, 200]), (3, 1, 128, [127, 128, 300]),
          (2, 8, 128, [40, 5, 0]), (1, 16, 256, [17, 70]), (2, 2, 192, [130, 3]), (1, 2, 96, [5, 97, 161]), (5, 1, 32, [255, 1, 1, 1, 2]),
          (4, 2, 128, [700]), (1, 1, 48, [1000])]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:3])))
@pytest.mark.parametrize("causal", [True, False])
def test_prompt(kind, shape, causal):
    heads, group, dim, n = shape
    gen = torch.Generator().manual_seed(dim + len(n))
    say(f"[gpu] {n} tokens")
    _prompt(*_qkv(gen, P.DT[kind], sum(n) + 5, sum(n) + 5, heads, group, dim), n, causal=causal)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_with_other_keys(kind, causal, dim):
    """More keys than tokens (a prefix), fewer (the first tokens see none), none at all."""
    gen = torch.Generator().manual_seed(dim)
    n, m = [10, 70, 33, 4, 0, 150], [100, 70, 0, 3, 9, 20]
    _prompt(*_qkv(gen, P.DT[kind], sum(n) + 3, sum(m) + 40, 2, 3, dim), n, m, causal)


@pytest.mark.parametrize("tokens", [1, 40, 1500])
def test_prompts_of_every_tile(tokens):
    """Few and many sequences and heads, so that tiles of each size are taken."""
    for batch, heads, group, dim in ((1, 1, 1, 64), (1, 8, 4, 128), (9, 4, 2, 64), (5, 8, 2, 256), (40, 16, 1, 64)):
        gen = torch.Generator().manual_seed(tokens + batch)
        n = [max(1, tokens * (i + 1) // batch // 4) for i in range(batch)]
        while sum(n) * heads * group > 60000:
            n = n[:-1] if len(n) > 1 else [n[0] // 2]
        say(f"[gpu] {n} tokens, {heads} x {group} heads of {dim}")
        _prompt(*_qkv(gen, torch.bfloat16, sum(n), sum(n), heads, group, dim), n)


def test_prompt_views():
    """Slices of a fused projection's rows, heads outermost, shared rows, an out with gaps."""
    gen = torch.Generator().manual_seed(3)
    heads, group, dim, n = 2, 3, 64, [70, 1, 130]
    total = sum(n)
    x = torch.randn(total + 2, (group + 2) * heads * dim + 64, generator=gen).to(torch.bfloat16)
    cut = lambda y: [z.unflatten(1, (-1, dim)) for z in (y[:, :group * heads * dim], y[:, group * heads * dim:(group + 1) * heads * dim],
                                                       y[:, (group + 1) * heads * dim:(group + 2) * heads * dim])]
    _prompt(*cut(x), n, devices=cut(x.cuda()))
    q, k, v = _qkv(gen, torch.float16, total, total, heads, group, dim)
    outer = lambda y: y.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    _prompt(q, k, v, n, devices=(outer(q), outer(k), outer(v)))
    one = k[:, :1].expand(-1, heads, -1)
    _prompt(q, one, v, n, devices=(q.cuda(), k.cuda()[:, :1].expand(-1, heads, -1), v.cuda()))
    row = k[:1].expand(total, -1, -1)
    _prompt(q, row, row, n, devices=(q.cuda(), k[:1].cuda().expand(total, -1, -1), k[:1].cuda().expand(total, -1, -1)))
    wide = torch.full((total, 2 * heads * group, dim + 16), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.zeros(heads * group, total + 1, device="cuda").t()[:total]
    out = wide[:, ::2, :dim]
    L.tc_prompt_attention(q.cuda(), k.cuda(), v.cuda(), _i32(R.starts_of(n)), out=out, lse=lse)
    ref = _prompt_ref(q, k, v, n, n, True)
    R.close(out, ref[0], ref[2], "out", q.dtype)
    R.close(lse, ref[1], ref[3], "lse")
    assert bool((wide[:, 1::2] == 7.0).all()) and bool((wide[..., dim:] == 7.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.0, 3.0])
def test_prompt_scales(kind, scale):
    gen = torch.Generator().manual_seed(4)
    _prompt(*_qkv(gen, P.DT[kind], 200, 200, 1, 2, 64, 1.0), [40, 160], scale=scale)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_ignores_what_is_not_seen(kind, bad, dim):
    """Infinities and NaN in the keys and values of later tokens, of other sequences and of padding; values in rows that are
    seen make their element infinite or NaN, in the rows that see them and no other."""
    gen = torch.Generator().manual_seed(5)
    n, heads, group = [90, 3, 150], 1, 2
    total = sum(n)
    q, k, v = _qkv(gen, P.DT[kind], total + 60, total + 60, heads, group, dim)
    good = _prompt_ref(q, k, v, n, n, True)
    k[total:], v[total:] = bad, bad
    v[60, 0, 5], k[92], v[92] = bad, bad, bad  # the last of sequence 1
    v[93 + 100, 0, 7:9] = bad
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    out, lse = torch.full_like(qd, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    L.tc_prompt_attention(qd, kd, vd, _i32(R.starts_of(n)), out=out, lse=lse)
    out, lse = out.cpu()[:total], lse.cpu()[:total]
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[60:90, :, 5] = True
    hit[92] = True
    hit[93 + 100:, :, 7:9] = True
    assert not bool(out[hit].isfinite().any())
    R.close(out[~hit], good[0][~hit], good[2][~hit], "out", q.dtype)
    rows = torch.ones(total, dtype=torch.bool)
    rows[92] = False
    R.close(lse[rows], good[1][rows], good[3][rows], "lse")


def test_prompt_keeps_the_sign_of_an_infinite_value():
    for first in (0, 40):
        q, k = (torch.zeros(64, 1, 32, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        v = torch.zeros_like(q)
        v[first, 0, 3], v[first, 0, 4], v[first, 0, 5] = math.inf, -math.inf, math.nan
        out = L.tc_prompt_attention(q, k, v, _i32([0, 64])).float()[:, 0]
        assert bool((out[first:, 3] == math.inf).all()) and bool((out[first:, 4] == -math.inf).all())
        assert bool(out[first:, 5].isnan().all())
        out[first:, 3:6] = 0
        assert bool((out == 0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_prompt_of_extreme_logits(kind):
    """Keys of the type's lowest value and of -infinity, maxima that grow from tile to tile and fall, far from zero."""
    dt, dim, n = P.DT[kind], 64, 400
    gen = torch.Generator().manual_seed(6)
    q, v = torch.zeros(n, 2, dim, dtype=dt), torch.randn(n, 1, dim, generator=gen).to(dt)
    q[:, :, 0] = 1.0
    low = torch.finfo(dt).min
    steps = torch.arange(n, dtype=torch.float32)
    for name, x in (("rise", steps / 4), ("fall", -steps / 4), ("far", 3000.0 + steps % 7), ("down", -3000.0 - steps % 5),
                    ("jumps", torch.where(steps % 90 == 89, steps, -steps)), ("low", torch.full((n,), low)),
                    ("one", torch.where(steps == 200, 0.0, torch.tensor(low)))):
        k = torch.zeros(n, 1, dim)
        k[:, 0, 0] = x
        say(f"[gpu] {name}")
        _prompt(q, k.to(dt), v, [n], scale=1.0)
    k = torch.zeros(n, 1, dim)
    k[:, 0, 0] = torch.where(steps < 150, -math.inf, steps / 50)
    out, lse, ref = _prompt(q, k.to(dt), v, [n], scale=1.0)
    assert bool((out[:150] == 0).all()) and bool((lse[:150] == -math.inf).all())


def test_prompt_of_many_light_rows_beside_a_heavy_one():
    """5000 weights of 2^-22 beside one of 1, where fp16 has subnormal numbers: they are not lost."""
    dim, n = 32, 5000
    q, k, v = (torch.zeros(x, 1, dim, dtype=torch.float16) for x in (1, n, n))
    q[:, 0, 0] = 1.0
    k[1:, 0, 0] = -22 * math.log(2.0)
    v[1:] = 100.0
    _prompt(q, k, v, [1], [n], scale=1.0)


def test_prompt_far_into_large_tensors():
    """Keys more than 2^32 bytes from the beginning."""
    tokens, heads, dim, pitch = 5000, 1, 64, 1 << 20
    gen = torch.Generator().manual_seed(7)
    base = torch.empty(tokens * (pitch // 2), dtype=torch.bfloat16, device="cuda")
    k, v = (base.as_strided((tokens, heads, dim), (pitch // 2, dim, 1), o) for o in (0, 4096))
    q, kh, vh = _qkv(gen, torch.bfloat16, 60, tokens, heads, 2, dim)
    k.copy_(kh), v.copy_(vh)
    _prompt(q, kh, vh, [0, 20, 40], [4200, 700, 100], devices=(q.cuda(), k, v))


def test_prompt_equal_calls_and_streams():
    gen = torch.Generator().manual_seed(8)
    n = [600, 33]
    q, k, v = (x.cuda() for x in _qkv(gen, torch.bfloat16, sum(n), sum(n), 2, 4, 128))
    starts = _i32(R.starts_of(n))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [L.tc_prompt_attention(q, k, v, starts, stream=x) for x in (None, s, s.cuda_stream)]
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert not L.tc_prompt_attention(q.detach().requires_grad_(), k, v, starts).requires_grad


# ---- over the cache --------------------------------------------------------------------------

def _random_masks(gen, n, kind):
    """Words for n tokens: a tree's ancestors, any bits, or none at all for some tokens."""
    words = []
    for i in range(n):
        if kind == "tree":
            up = int(torch.randint(-1, max(1, i), (1,), generator=gen)) if i else -1
            words.append((words[up] if up >= 0 else 0) | (1 << i if i < 64 else 0))
        elif kind == "empty":
            words.append(0 if i % 3 else 1 << i % 64)
        else:
            hi, lo = torch.randint(0, 2 ** 32, (2,), generator=gen).tolist()
            words.append(hi << 32 | lo)
    return words


def _tree_ref(q, pool, table, lens, n, page, words, scale=None, part=None):
    parts, a = [], 0
    for b, t in enumerate(n):
        m = lens[b]
        k, ok = pool.rows("k", table[b], m, page)
        v, _ = pool.rows("v", table[b], m, page)
        seen = R.before(t, m) if words is None else R.by_masks(words[a:a + t], t, m)
        kind = torch.bfloat16 if pool.kind == "e4m3" else P.DT[pool.kind]
        ref = R.sequence(q[a:a + t], k, v, seen & ok[None, :], scale,
                         R.half_step(kind) if part is None else part)
        parts.append(ref)
        a += t
    return [torch.cat(p) for p in zip(*parts)]


def _tree(q, pool, table, lens, n, page, words=None, scale=None, max_len=None, cache=None):
    cache = pool.on_gpu() if cache is None else cache
    qd = q.cuda()
    out, lse = torch.full_like(qd, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    masks = None if words is None else _i64(words + [2 ** 64 - 1] * (q.shape[0] - len(words)))
    got = L.tc_paged_tree_attention(qd, cache, table.cuda(), _i32(lens), _i32(R.starts_of(n)), masks=masks, scale=scale,
                                    max_len=max_len, out=out, lse=lse)
    torch.cuda.synchronize()
    assert got is out
    ref = _tree_ref(q, pool, table, lens, n, page, words, scale)
    total = sum(n)
    R.close(out[:total], ref[0], ref[2] + _fp16_subnormals(q, pool, ref), "out", q.dtype)
    R.close(lse[:total], ref[1], ref[3], "lse")
    assert bool((out[total:] == 7.0).all()) and bool((lse[total:] == 7.0).all())
    return out, lse, ref


def _fp16_subnormals(q, pool, ref):
    """2^-32 of a row's greatest weight (at most 1) for each of its rows' values, where weights are fp16."""
    return 2.0 ** -32 * 5.0 * 20000 if pool.kind == "fp16" else 0.0


TREES = [  # heads, group, dim, page, major, lens, tokens
    (1, 1, 16, 16, "rows", [1], [1]),
    (2, 4, 64, 16, "heads", [100, 7, 0, 40], [8, 7, 0, 1]),
    (1, 3, 80, 7, "rows", [65, 129, 64], [5, 64, 33]),
    (2, 2, 128, 24, "rows", [700, 300], [20, 16]),
    (1, 8, 128, 16, "pairs", [1000, 513], [12, 64]),
    (1, 4, 256, 1, "rows", [90, 33], [9, 3]),
    (2, 2, 192, 100, "heads", [600], [30]),
    (4, 1, 128, 64, "heads", [1, 64, 65], [1, 1, 2]),
    (1, 2, 64, 4, "rows", [3000], [40]),
    (2, 8, 64, 32, "rows", [2100, 5], [60, 4]),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"])
@pytest.mark.parametrize("shape", TREES, ids=lambda s: "x".join(map(str, s[:4])))
@pytest.mark.parametrize("mask", ["tree", "any", "empty", None])
def test_tree(kind, shape, mask):
    heads, group, dim, page, major, lens, n = shape
    kinds = kind.split("-")
    gen = torch.Generator().manual_seed(dim + page)
    table, pages = P.table_for(lens, page, gen, spare=1)
    pool = P.Pool(kinds[-1], pages, page, heads, dim, major, gen)
    q = (2.5 * torch.randn(sum(n) + 3, heads * group, dim, generator=gen)).to(P.DT[kinds[0]])
    words = None if mask is None else [w for t in n for w in _random_masks(gen, t, mask)]
    say(f"[gpu] {n} tokens over {lens} rows")
    _tree(q, pool, table, lens, n, page, words)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3"])
def test_more_tokens_than_words_have_bits(kind):
    """With masks, tokens from the 65th on are seen by none; chunks of a prompt see all before them."""
    kinds = kind.split("-")
    gen = torch.Generator().manual_seed(9)
    lens, n, page = [500, 90, 70], [200, 66, 70], 16
    table, pages = P.table_for(lens, page, gen)
    pool = P.Pool(kinds[-1], pages, page, 2, 64, "rows", gen)
    q = torch.randn(sum(n), 4, 64, generator=gen).to(P.DT[kinds[0]])
    _tree(q, pool, table, lens, n, page)
    _tree(q, pool, table, lens, n, page, [w for t in n for w in _random_masks(gen, t, "tree")])


def test_fewer_rows_than_tokens():
    """Tokens whose rows would lie before a sequence's first: they see what exists of what they name."""
    gen = torch.Generator().manual_seed(10)
    lens, n, page = [3, 0, 40], [9, 4, 50], 16
    table, pages = P.table_for(lens, page, gen)
    pool = P.Pool("bf16", pages, page, 1, 64, "rows", gen)
    q = torch.randn(sum(n), 2, 64, generator=gen).to(torch.bfloat16)
    out, lse, _ = _tree(q, pool, table, lens, n, page)
    assert bool((out[:6] == 0).all()) and bool((lse[9:13] == -math.inf).all())
    _tree(q, pool, table, lens, n, page, [w for t in n for w in _random_masks(gen, t, "any")])


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("page", [16, 5])
def test_tree_ignores_missing_pages_and_what_is_not_seen(kind, page):
    """Pages that are none, NaN in pages of no sequence, in rows past the end and in drafted rows that a token does not see."""
    gen = torch.Generator().manual_seed(11)
    lens, n, heads, dim = [700, 150], [10, 7], 2, 64
    dt = torch.bfloat16 if kind == "e4m3" else P.DT[kind]
    table, pages = P.table_for(lens, page, gen, spare=1, junk=10 ** 6)
    pool = P.Pool(kind, pages, page, heads, dim, "rows", gen)
    spare = ({*range(pages)} - {int(x) for x in table.flatten().tolist() if x < pages}).pop()
    q = torch.randn(sum(n), 4, dim, generator=gen).to(dt)
    words = [w for t in n for w in _random_masks(gen, t, "tree")]
    for w in range(len(words)):
        words[w] &= ~(1 << 3)  # the fourth token of each sequence is seen by none
    table[0, 2], table[0, 11], table[1, 0] = -1, pages, 2 ** 31 - 1
    good = _tree_ref(q, pool, table, lens, n, page, words)
    where = [(int(table[b, (m - t + 3) // page]), (m - t + 3) % page) for b, (m, t) in enumerate(zip(lens, n))]
    where += [(int(table[b, (m - 1) // page]), r) for b, m in enumerate(lens) for r in range((m - 1) % page + 1, page)]
    where += [(spare, r) for r in range(page)]
    for g, r in where:
        for x in (pool.k, pool.v):
            P.bits(x)[g, r] = P.bits(torch.full((1,), math.nan).to(x.dtype))[0]
        if pool.ks is not None:
            pool.ks[g, r], pool.vs[g, r] = math.nan, math.inf
    qd = q.cuda()
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = L.tc_paged_tree_attention(qd, pool.on_gpu(), table.cuda(), _i32(lens), _i32(R.starts_of(n)), masks=_i64(words), lse=lse)
    R.close(out, good[0], good[2] + _fp16_subnormals(q, pool, good), "out", dt)
    R.close(lse, good[1], good[3], "lse")


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
def test_tree_of_nan_values_that_are_seen(kind):
    gen = torch.Generator().manual_seed(12)
    lens, n, page, dim = [200], [6], 16, 64
    dt = torch.bfloat16 if kind == "e4m3" else P.DT[kind]
    table, pages = P.table_for(lens, page, gen)
    pool = P.Pool(kind, pages, page, 1, dim, "rows", gen)
    q = torch.randn(6, 2, dim, generator=gen).to(dt)
    words = [1 << i for i in range(6)]
    good = _tree_ref(q, pool, table, lens, n, page, words)
    P.bits(pool.v)[int(table[0, 197 // page]), 197 % page, 0, 9] = P.bits(torch.full((1,), math.nan).to(pool.v.dtype))[0]
    out = L.tc_paged_tree_attention(q.cuda(), pool.on_gpu(), table.cuda(), _i32(lens), _i32([0, 6]), masks=_i64(words)).cpu()
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[3, :, 9] = True
    assert bool(out[hit].isnan().all())
    R.close(out[~hit], good[0][~hit], (good[2] + _fp16_subnormals(q, pool, good))[~hit], "out", dt)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3"])
@pytest.mark.parametrize("batch, length, tokens, heads, group, dim", [
    (1, 20000, 3, 1, 2, 64), (2, 9000, 12, 2, 8, 128), (1, 6000, 64, 1, 8, 128), (70, 600, 2, 4, 1, 64), (3, 5000, 9, 2, 4, 256),
    (130, 513, 1, 1, 1, 32)])
def test_tree_over_split_caches(kind, batch, length, tokens, heads, group, dim):
    """Long caches of unequal lengths, whose tiles are split and joined."""
    kinds = kind.split("-")
    gen = torch.Generator().manual_seed(length)
    lens = [max(tokens, length * (i + 1) // batch) for i in range(batch)]
    lens[batch // 2] = 0 if batch > 2 else lens[batch // 2]
    n = [min(tokens, m) for m in lens]
    table, pages = P.table_for(lens, 16, gen)
    pool = P.Pool(kinds[-1], pages, 16, heads, dim, "rows", gen)
    q = torch.randn(sum(n), heads * group, dim, generator=gen).to(P.DT[kinds[0]])
    words = [w for t in n for w in _random_masks(gen, t, "tree")]
    need = L.load_library().tc_paged_tree_attention_workspace(batch, sum(n), heads * group, heads, dim, max(lens))
    assert need > 0
    say(f"[gpu] {batch} sequences of up to {length} rows")
    out, lse, _ = _tree(q, pool, table, lens, n, 16, words, max_len=max(lens))
    again, _, _ = _tree(q, pool, table, lens, n, 16, words, max_len=max(lens))
    assert torch.equal(out, again)


def test_a_tree_of_one_token_is_the_attention_of_one_token():
    gen = torch.Generator().manual_seed(13)
    lens, page = [300, 5000, 1, 0], 16
    for kind in ("bf16", "fp16", "e4m3"):
        dt = torch.bfloat16 if kind == "e4m3" else P.DT[kind]
        table, pages = P.table_for(lens, page, gen)
        pool = P.Pool(kind, pages, page, 2, 128, "rows", gen)
        cache = pool.on_gpu()
        q = torch.randn(4, 8, 128, generator=gen).to(dt)
        a, b = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
        one = L.tc_paged_attention(q.cuda(), cache, table.cuda(), _i32(lens), lse=a)
        for masks in (None, _i64([1] * 4)):
            many = L.tc_paged_tree_attention(q.cuda(), cache, table.cuda(), _i32(lens), _i32(range(5)), masks=masks, lse=b)
            ref = _tree_ref(q, pool, table, lens, [1] * 4, page, None)
            R.close(many, one.cpu().double(), 2 * ref[2] + torch.finfo(dt).eps * ref[0].abs() + _fp16_subnormals(q, pool, ref), "out", dt)
            R.close(b, a.cpu().double(), 2 * ref[3], "lse")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 3])
def test_tree_far_into_a_large_pool(kind, page):
    """Rows more than 2^32 bytes from the pool's beginning, and pages more than 2^31 elements apart."""
    heads, dim, batch, length = 1, 64, 2, 100
    cols = -(-length // page)
    pitch = (1 << 32) // (batch * cols) // 16 * 16 + (1 << 20)  # elements from page to page
    dt = P.DT[kind]
    pages = batch * cols
    gen = torch.Generator().manual_seed(14)
    x = torch.empty(pages * pitch * dt.itemsize, dtype=torch.uint8, device="cuda")
    small = P.Pool(kind, pages, page, heads, dim, "rows", gen)
    at = x.view(dt)
    k, v = (at.as_strided((pages, page, heads, dim), (pitch, heads * dim, dim, 1), o) for o in (0, 1 << 17))
    P.bits(k).copy_(P.bits(small.k)), P.bits(v).copy_(P.bits(small.v))
    cache = L.PagedCache(k, v, *(None if s is None else s.cuda() for s in (small.ks, small.vs)))
    table = torch.randperm(pages, generator=gen).to(torch.int32).view(batch, cols)
    q = torch.randn(12, 4, dim, generator=gen).to(torch.bfloat16)
    _tree(q, small, table, [length, length - 7], [5, 7], page, cache=cache)


def test_tree_views():
    """q and out as slices, a table with strides, a max_len below a sequence's length."""
    gen = torch.Generator().manual_seed(15)
    lens, n, page = [90, 40], [5, 8], 16
    table, pages = P.table_for(lens, page, gen)
    pool = P.Pool("fp16", pages, page, 2, 64, "heads", gen)
    wide = torch.randn(13, 12, 64, generator=gen).to(torch.float16)
    q = wide[:, 4:8]
    t = torch.zeros(table.shape[1], 4, dtype=torch.int32, device="cuda").t()[::2]
    t.copy_(table)
    into = torch.full((13, 8, 80), 7.0, dtype=torch.float16, device="cuda")
    out = into[:, ::2, :64]
    L.tc_paged_tree_attention(wide.cuda()[:, 4:8], pool.on_gpu(), t, _i32(lens), _i32([0, 5, 13]), out=out)
    ref = _tree_ref(q, pool, table, lens, n, page, None)
    R.close(out, ref[0], ref[2] + _fp16_subnormals(q, pool, ref), "out", q.dtype)
    assert bool((into[:, 1::2] == 7.0).all()) and bool((into[..., 64:] == 7.0).all())
    got = L.tc_paged_tree_attention(q.cuda(), pool.on_gpu(), t, _i32(lens), _i32([0, 5, 13]), max_len=60)
    ref = _tree_ref(q, pool, table, [60, 40], n, page, None)
    R.close(got, ref[0], ref[2] + _fp16_subnormals(q, pool, ref), "out", q.dtype)


def test_calls_from_threads_on_separate_streams():
    jobs, errors = [], []
    for i in range(6):
        gen = torch.Generator().manual_seed(90 + i)
        lens, n = [50 * i + 30, 2900 - 100 * i, 17], [9, 20, 3]
        table, pages = P.table_for(lens, 16, gen)
        kind = ("bf16", "fp16", "e4m3")[i % 3]
        pool = P.Pool(kind, pages, 16, 2, 64, "rows", gen)
        q = torch.randn(sum(n), 8, 64, generator=gen).to(torch.float16 if i % 3 == 1 else torch.bfloat16)
        ref = _tree_ref(q, pool, table, lens, n, 16, None)
        jobs.append((pool.on_gpu(), q.cuda(), table.cuda(), _i32(lens), _i32(R.starts_of(n)), ref, _fp16_subnormals(q, pool, ref)))
    torch.cuda.synchronize()

    def work(cache, q, table, lens, starts, ref, more):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(8):
                    out = L.tc_paged_tree_attention(q, cache, table, lens, starts, max_len=3000)
                    with pytest.raises(L.TileCopyError):
                        L.tc_paged_tree_attention(q, cache, table, lens, starts, max_len=-1)
                    s.synchronize()
                    R.close(out, ref[0], ref[2] + more, "out", q.dtype)
        except BaseException as e:  # reported below
            errors.append(repr(e))

    say(f"[gpu] {len(jobs)} threads")
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:2]


def test_captured_calls_replay_with_new_contents():
    """A prompt's and a tree's attention captured once, on a stream of their own each, and replayed while lengths, starts,
    tables, masks and tokens move on, with the program's own work between the replays."""
    gen = torch.Generator().manual_seed(16)
    heads, group, dim, page, batch, cols, room = 2, 4, 128, 16, 3, 80, 96
    pages = batch * cols
    pool = P.Pool("bf16", pages, page, heads, dim, "rows", gen)
    cache = pool.on_gpu()
    table = torch.randperm(pages, generator=gen).to(torch.int32).view(batch, cols)
    t_d, lens_d, starts_d = table.cuda(), _i32([0] * batch), _i32([0] * (batch + 1))
    q_d = torch.zeros(room, heads * group, dim, device="cuda", dtype=torch.bfloat16)
    k_d, v_d = (torch.zeros(room, heads, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    masks_d = torch.zeros(room, dtype=torch.int64, device="cuda")
    graphs = []
    for which in range(3):
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        lse = torch.zeros(room, heads * group, device="cuda")
        out = torch.zeros_like(q_d)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            if which:
                L.tc_paged_tree_attention(q_d, cache, t_d, lens_d, starts_d, masks=masks_d if which == 1 else None, out=out, lse=lse)
            else:
                L.tc_prompt_attention(q_d, k_d, v_d, starts_d, out=out, lse=lse)
        graphs.append((g, out, lse, s))
    for step, (lens, n) in enumerate([([50, 1280, 7], [20, 40, 7]), ([900, 0, 64], [64, 0, 32]), ([1, 2, 3], [1, 1, 1]),
                                      ([1280, 1280, 1280], [32, 32, 32]), ([5, 600, 70], [0, 3, 60])]):
        q = torch.randn(room, heads * group, dim, generator=gen).to(torch.bfloat16)
        k, v = (torch.randn(room, heads, dim, generator=gen).to(torch.bfloat16) for _ in range(2))
        words = [w for t in n for w in _random_masks(gen, t, "tree")]
        q_d.copy_(q), k_d.copy_(k), v_d.copy_(v), lens_d.copy_(_i32(lens)), starts_d.copy_(_i32(R.starts_of(n)))
        masks_d.copy_(_i64(words + [0] * (room - len(words))))
        (torch.randn(1 << 20, device="cuda") * 2).sum().item()
        torch.cuda.synchronize()
        for g, _, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        say(f"[gpu] replay {step}")
        refs = [_prompt_ref(q, k, v, n, n, True), _tree_ref(q, pool, table, lens, n, page, words),
                _tree_ref(q, pool, table, lens, n, page, None)]
        for (_, out, lse, _), ref in zip(graphs, refs):
            R.close(out[:sum(n)], ref[0], ref[2], "out", q.dtype)
            R.close(lse[:sum(n)], ref[1], ref[3], "lse")


def test_empty_calls():
    e = lambda *s, **k: torch.zeros(*s, device="cuda", **k)
    h = dict(dtype=torch.bfloat16)
    L.tc_prompt_attention(e(0, 4, 64, **h), e(0, 2, 64, **h), e(0, 2, 64, **h), _i32([0]))
    L.tc_prompt_attention(e(0, 4, 64, **h), e(0, 2, 64, **h), e(0, 2, 64, **h), _i32([0, 0]))
    out = torch.full((3, 4, 64), 7.0, device="cuda", **h)
    L.tc_prompt_attention(e(3, 4, 64, **h), e(3, 2, 64, **h), e(3, 2, 64, **h), _i32([0]), out=out)
    assert bool((out == 7.0).all())
    lse = e(3, 4)
    L.tc_prompt_attention(e(3, 4, 64, **h), e(0, 2, 64, **h), e(0, 2, 64, **h), _i32([0, 2]), key_starts=_i32([0, 0]), out=out, lse=lse)
    assert bool((out[:2] == 0).all()) and bool((out[2] == 7.0).all()) and bool((lse[:2] == -math.inf).all())
    pool = P.Pool("bf16", 4, 16, 2, 64, "rows", fill=1.0)
    cache = pool.on_gpu()
    table = _i32([[0, 1], [2, 3]])
    L.tc_paged_tree_attention(e(0, 4, 64, **h), cache, table, _i32([5, 6]), _i32([0, 0, 0]))
    out.fill_(7.0)
    L.tc_paged_tree_attention(e(3, 4, 64, **h), cache, table, _i32([5, 6]), _i32([0, 0, 2]), out=out)
    assert bool((out[:2] == 1).all()) and bool((out[2] == 7.0).all())
    L.tc_paged_tree_attention(e(3, 4, 64, **h), cache, _i32([]).view(0, 2), _i32([]), _i32([0]), out=out)
    L.tc_paged_tree_attention(e(2, 4, 64, **h), cache, _i32([]).view(2, 0), _i32([5, 6]), _i32([0, 1, 2]), out=out[:2])
    assert bool((out[:2] == 0).all())
    none = L.PagedCache(e(0, 16, 2, 64, **h), e(0, 16, 2, 64, **h))
    out.fill_(7.0)
    L.tc_paged_tree_attention(e(2, 4, 64, **h), none, table, _i32([5, 6]), _i32([0, 1, 2]), out=out[:2])
    assert bool((out[:2] == 0).all()) and bool((out[2] == 7.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [80, 128, 144, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_in_the_largest_tiles(kind, dim, causal):
    """Enough rows and heads for tiles of 256 rows; all heads are copies of two, and equal to them."""
    n, heads = [2900, 1200], 32
    gen = torch.Generator().manual_seed(dim)
    q, k, v = _qkv(gen, P.DT[kind], sum(n), sum(n), 2, 1, dim)
    which = torch.arange(heads) % 2
    starts = _i32(R.starts_of(n))
    out = L.tc_prompt_attention(q.cuda()[:, which], k.cuda()[:, which], v.cuda()[:, which], starts, causal=causal)
    ref = _prompt_ref(q, k, v, n, n, causal)
    for h in (0, 1):
        R.close(out[:, h], ref[0][:, h], ref[2][:, h], "out", q.dtype)
        assert torch.equal(out[:, h::2], out[:, h:h + 1].expand(-1, heads // 2, -1))


LARGE = [  # heads, group, dim, page, major, lens, tokens (causal chunks)
    (2, 1, 128, 24, "rows", [900, 300], [400, 257]), (1, 2, 96, 5, "heads", [513, 700], [130, 300]),
    (1, 4, 256, 16, "rows", [600], [90]), (1, 2, 192, 7, "pairs", [300, 1400], [300, 129]), (2, 4, 128, 64, "heads", [640], [64])]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"])
@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s[:4])))
def test_tree_in_the_largest_tiles(kind, shape):
    """Sequences of 256 query rows and more, one page of each missing: chunks of prompts, and with masks."""
    heads, group, dim, page, major, lens, n = shape
    kinds = kind.split("-")
    gen = torch.Generator().manual_seed(dim + page)
    table, pages = P.table_for(lens, page, gen, spare=1)
    for b, m in enumerate(lens):
        table[b, (m // 2) // page] = -1
    pool = P.Pool(kinds[-1], pages, page, heads, dim, major, gen)
    q = torch.randn(sum(n), heads * group, dim, generator=gen).to(P.DT[kinds[0]])
    say(f"[gpu] {n} tokens over {lens} rows")
    _tree(q, pool, table, lens, n, page)
    words = [w for t in n for w in _random_masks(gen, t, "any")]
    _tree(q, pool, table, lens, n, page, words)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads, group, dim, n, m", [
    (1, 4, 64, [5, 0, 40], [4000, 0, 1200]), (2, 1, 128, [1], [5001]), (2, 8, 128, [17, 20], [1, 4096]), (1, 2, 256, [70, 3, 0], [3001, 2000, 7]),
    (3, 1, 96, [200], [1700]), (1, 1, 192, [9] * 70, [1600] * 70)])
def test_prompts_of_few_queries_and_long_keys(kind, causal, heads, group, dim, n, m):
    """Tiles split over their keys and joined; more sequences than lanes; the same bits again."""
    gen = torch.Generator().manual_seed(dim + len(n))
    need = L.load_library().tc_prompt_attention_workspace(len(n), sum(n) + 3, sum(m) + 40, heads * group, heads, dim)
    assert need > 0
    say(f"[gpu] {n[:3]} tokens over {m[:3]} keys, {need} bytes")
    q, k, v = _qkv(gen, P.DT[kind], sum(n) + 3, sum(m) + 40, heads, group, dim)
    k[sum(m):], v[sum(m):] = math.nan, math.nan
    out, lse, _ = _prompt(q, k, v, n, m, causal)
    again, lse_again, _ = _prompt(q, k, v, n, m, causal)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


def test_starts_that_do_not_ascend_stay_inside():
    """What such a call leaves is its own affair; it ends, keeps to its tensors, and the next one is right."""
    gen = torch.Generator().manual_seed(21)
    q, k, v = _qkv(gen, torch.bfloat16, 96, 8000, 1, 4, 64)
    back = _i32([0, 96, 0, 96, 0, 96, 0, 96, -5, 200])
    around = torch.full((3, 96, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    L.tc_prompt_attention(q.cuda(), k.cuda(), v.cuda(), back, key_starts=_i32([0, 8000, 0, 8000, 9000, 8000, -3, 8000, 1, 8000]), out=around[1])
    pool = P.Pool("bf16", 500, 16, 1, 64, "rows", gen)
    table = torch.arange(500, dtype=torch.int32).reshape(1, 500).expand(9, 500).contiguous()
    L.tc_paged_tree_attention(q.cuda(), pool.on_gpu(), table.cuda(), _i32([8000] * 9), back, out=around[1])
    assert bool((around[0] == 7.0).all()) and bool((around[2] == 7.0).all())
    _prompt(q, k, v, [96], [8000])
    _tree(q, pool, table[:1], [8000], [96], 16)


@pytest.mark.parametrize("shape", LARGE + TREES[:5], ids=lambda s: "x".join(map(str, s[:4])))
def test_fp16_over_8_bit_rows_keeps_its_bits(shape):
    """Weights there are the sum of two bf16 values, off by the square of half a bf16 step (2^-8), in tiles of every size."""
    heads, group, dim, page, major, lens, n = shape
    gen = torch.Generator().manual_seed(dim + page)
    table, pages = P.table_for(lens, page, gen, spare=1)
    pool = P.Pool("e4m3", pages, page, heads, dim, major, gen)
    q = torch.randn(sum(n), heads * group, dim, generator=gen).to(torch.float16)
    out, _, _ = _tree(q, pool, table, lens, n, page)
    ref = _tree_ref(q, pool, table, lens, n, page, None, part=2.0 ** -16)
    R.close(out, ref[0], ref[2], "out", torch.float16)
