"""Attention of several query rows at the ends of its ranges: values near the end of fp32's, logits far from zero, many
sequences."""

import random
import time

import pytest
import torch

import layout_permuting_copy_amd as L
import paged_ref as P
import rows_ref as R
from gpu_util import say
from test_gpu_rows import _prompt, _prompt_ref, _random_masks, _tree

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
        pool.vs[at, row] = v.abs().amax(-1) / 2048  # 2^119 is promised there
    else:
        pool.k[at, row], pool.v[at, row] = k, v.to(torch.bfloat16)
    say(f"[gpu] {tokens} tokens over {rows} rows of {dim}")
    for words in (None, _random_masks(gen, tokens, "tree")):
        out, _, ref = _tree(q, pool, table, [rows], [tokens], 16, words, scale=1.0, max_len=rows)
        assert bool(out.isfinite().all()) and float(ref[0].abs().max()) > (1e36 if kind == "bf16" else 1e33) / rows


@pytest.mark.parametrize("exponent", [-126, -118, -110, 0, 118])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim, tokens, rows", [(64, 5, 300), (128, 70, 300), (256, 5, 4000)])
def test_tree_scales_of_either_end(exponent, dtype, dim, tokens, rows):
    """Scales from the least normal number to near the greatest that are promised to work, under a maximum that grows slower
    than what the reference follows, with codes of one sign: nothing overflows, and no bits are lost but those that numbers below
    2^-126 have not: of weights times scales (half of 2^-133 each, times a code of 448, the sum of weights being at least 1) and
    of out."""
    gen = torch.Generator().manual_seed(dim)
    table, pages = P.table_for([rows], 16, gen)
    pool = P.Pool("e4m3", pages, 16, 1, dim, "rows", gen)
    q, k, _ = _rising(rows, 1, dim, tokens, 2, rows // 15, gen)
    q = q.to(P.DT[dtype])
    at, row = table[0][torch.arange(rows) // 16].long(), torch.arange(rows) % 16
    P.bits(pool.k)[at, row] = P.bits(k.float().sign().to(torch.float8_e4m3fn))
    pool.ks[at, row] = k.float().amax(-1)
    most = 14.0 / rows if exponent > 100 else 448.0  # sums of all rows stay below 2^119
    P.bits(pool.v)[at, row] = P.bits((torch.rand(rows, 1, dim, generator=gen) * most / 2 + most / 2).to(torch.float8_e4m3fn))
    pool.vs.fill_(2.0 ** exponent)
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")
    out = L.tc_paged_tree_attention(q.cuda(), pool.on_gpu(), table.cuda(), i32([rows]), i32([0, tokens]), scale=1.0, max_len=rows)
    say(f"[gpu] scales of 2^{exponent}")
    if dtype == "fp16" and exponent > 0:
        assert bool((out == torch.inf).all())  # past fp16's own range
        return
    kr, vr = (pool.rows(x, table[0], rows, 16)[0] for x in "kv")
    ref = R.sequence(q, kr, vr, R.before(tokens, rows), 1.0, 2.0 ** -8)
    lost = 2.0 ** -134 * 448 * rows + (2.0 ** -134 if dtype == "bf16" else 2.0 ** -25)
    assert bool(out.isfinite().all())
    R.close(out, ref[0], ref[2] + lost, "out", q.dtype)


def _far(kind, x, rows, tokens, dim, gen):
    """Keys whose logits (scale 1) are exactly x where queries see them, and the definition with x taken off all of them, whose
    weights are the same: bounds without the logits' own rounding, of which there is none."""
    dt = torch.bfloat16 if kind == "e4m3" else P.DT[kind]
    most = 1.0 if kind == "e4m3" else 2.0 ** 14 if kind == "fp16" else 1.0
    q, k = torch.zeros(tokens, 2, dim, dtype=torch.float32), torch.zeros(rows, 1, dim)
    q[:, :, 0], k[:, :, 0] = most, (x / most)[:, None]
    assert bool((q.to(dt).double()[:1, 0, 0] * k.to(dt).double()[:, 0, 0] == x.double()).all())
    v = torch.randn(rows, 1, dim, generator=gen).to(dt)
    return q.to(dt), k.to(dt), v


FAR = [(kind, x) for kind in ("bf16", "fp16") for x in (2.0 ** 24, 3 * 2.0 ** 26, 5 * 2.0 ** 25, -5 * 2.0 ** 25, -1.75 * 2.0 ** 28, 2.0 ** 28, -7 * 2.0 ** 26)]
FAR += [("bf16", x) for x in (-1.5 * 2.0 ** 33, 2.0 ** 40, -1.25 * 2.0 ** 63, 1.25 * 2.0 ** 63, -2.0 ** 100, 1.75 * 2.0 ** 99, -1.25 * 2.0 ** 126, 2.0 ** 127)]


@pytest.mark.parametrize("kind, x", FAR)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_logits_far_from_zero(kind, x, dim):
    """Equal logits share the weight, a greater one has it all, wherever they lie; a rise to x comes in the middle."""
    gen = torch.Generator().manual_seed(3)
    n = 200
    levels = torch.full((n,), x)
    for name, xs in (("equal", levels), ("rise", torch.where(torch.arange(n) < 100, 0.5 * levels if x > 0 else 2 * levels, levels)),
                     ("few", torch.where(torch.arange(n) % 67 == 5, levels, 0.5 * levels if x > 0 else 2 * levels))):
        if not bool(xs.isfinite().all()):
            continue
        q, k, v = _far(kind, xs, n, n, dim, gen)
        seen = R.before(n, n)
        top = torch.where(seen, xs[None, :], -torch.inf).amax(1)
        flat = torch.zeros_like(k)
        ref = R.sequence(q, flat, v, seen & (xs[None, :] == top[:, None]))  # the others' weights are 0 in any precision
        out, lse = torch.zeros_like(q, device="cuda"), torch.zeros(n, 2, device="cuda")
        say(f"[gpu] {name} {x}")
        L.tc_prompt_attention(q.cuda(), k.cuda(), v.cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale=1.0, out=out, lse=lse)
        R.close(out, ref[0], ref[2], "out", q.dtype)
        want = ref[1] + top[:, None].double()
        R.close(lse, want, ref[3] + 4 * R.STEP32 * want.abs(), "lse")


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("x", [5 * 2.0 ** 25, -5 * 2.0 ** 25, -7 * 2.0 ** 26])
@pytest.mark.parametrize("rows", [90, 2500])
def test_tree_logits_far_from_zero(kind, x, rows):
    """Equal logits over a cache, whole and in parts; 8-bit rows by their scales."""
    gen = torch.Generator().manual_seed(4)
    tokens, dim = 6, 64
    table, pages = P.table_for([rows], 16, gen)
    pool = P.Pool(kind, pages, 16, 1, dim, "rows", gen)
    q, k, v = _far(kind, torch.full((rows,), x), rows, tokens, dim, gen)
    at, row = table[0][torch.arange(rows) // 16].long(), torch.arange(rows) % 16
    if kind == "e4m3":
        P.bits(pool.k)[at, row] = P.bits(torch.zeros_like(k, dtype=torch.float32).to(torch.float8_e4m3fn))
        P.bits(pool.k)[at, row, :, 0] = P.bits(torch.ones(1).to(torch.float8_e4m3fn))[0]
        pool.ks[at, row] = x
        v = pool.rows("v", table[0], rows, 16)[0]
    else:
        pool.k[at, row], pool.v[at, row] = k, v
    seen = R.before(tokens, rows)
    part = None if kind != "e4m3" else R.half_step(torch.bfloat16)
    ref = R.sequence(q, torch.zeros_like(k), v, seen, part=part)
    lse = torch.zeros(tokens, 2, device="cuda")
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")
    out = L.tc_paged_tree_attention(q.cuda(), pool.on_gpu(), table.cuda(), i32([rows]), i32([0, tokens]), scale=1.0, lse=lse, max_len=rows)
    R.close(out, ref[0], ref[2], "out", q.dtype)
    R.close(lse, ref[1] + x, ref[3] + 4 * R.STEP32 * abs(x), "lse")


def _counts(pattern, batch):
    """Tokens of each sequence: some of none, some of more than a tile."""
    rng = random.Random(f"{pattern} {batch}")
    few = {"ones": lambda i: 1, "sparse": lambda i: 3 if i % 41 == 7 else 0, "ragged": lambda i: rng.choice([0, 0, 1, 2, 5, 13]),
           "one long": lambda i: 300 if i == batch // 2 else i % 2, "last": lambda i: 70 * (i == batch - 1), "first": lambda i: 70 * (i == 0),
           "none": lambda i: 0}
    return [few[pattern](i) for i in range(batch)]


MANY = [(p, b) for p in ("ones", "sparse", "ragged", "one long", "last", "first", "none") for b in (65, 2500)] + [("ragged", 1000), ("sparse", 5000)]


@pytest.mark.parametrize("pattern, batch", MANY)
@pytest.mark.parametrize("heads, group, dim, lead", [(2, 5, 64, 75), (1, 1, 256, 0)])
def test_prompts_of_many_sequences(pattern, batch, heads, group, dim, lead):
    """Tokens before the first sequence and behind the last belong to none, and stay as they are."""
    gen = torch.Generator().manual_seed(batch)
    n = _counts(pattern, batch)
    total, tokens = sum(n), lead + sum(n) + 9
    dt = torch.bfloat16 if batch % 2 else torch.float16
    q, k, v = (torch.randn(tokens, h, dim, generator=gen).to(dt) for h in (heads * group, heads, heads))
    starts = torch.tensor([lead + x for x in R.starts_of(n)], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0, device="cuda"), torch.full((tokens, heads * group), 7.0, device="cuda")
    say(f"[gpu] {batch} sequences, {total} tokens")
    L.tc_prompt_attention(q.cuda(), k.cuda(), v.cuda(), starts, out=out, lse=lse)
    if total:
        at = slice(lead, lead + total)
        ref = _prompt_ref(q[at], k[at], v[at], n, n, True)
        R.close(out[at], ref[0], ref[2], "out", dt)
        R.close(lse[at], ref[1], ref[3], "lse")
    rest = torch.ones(tokens, dtype=torch.bool)
    rest[lead:lead + total] = False
    assert bool((out[rest.cuda()] == 7.0).all()) and bool((lse[rest.cuda()] == 7.0).all())


@pytest.mark.parametrize("pattern, batch", [(p, b) for p, b in MANY if b < 3000])
@pytest.mark.parametrize("heads, group, dim", [(1, 4, 64), (1, 1, 192)])
def test_trees_of_many_sequences(pattern, batch, heads, group, dim):
    gen = torch.Generator().manual_seed(batch)
    n = _counts(pattern, batch)
    lens = [max(x, (37 * i) % 50 + (x > 0) * (i % 3 == 0) * 90) for i, x in enumerate(n)]
    table, pages = P.table_for(lens, 16, gen)
    pool = P.Pool("bf16", pages, 16, heads, dim, "rows", gen)
    q = torch.randn(sum(n) + 5, heads * group, dim, generator=gen).to(torch.bfloat16)
    say(f"[gpu] {batch} sequences, {sum(n)} tokens")
    if sum(n):
        _tree(q, pool, table, lens, n, 16, max_len=max(lens))
        _tree(q, pool, table, lens, n, 16, [w for t in n for w in _random_masks(gen, t, "tree")], max_len=max(lens))
    else:
        out = torch.full_like(q, 7.0, device="cuda")
        L.tc_paged_tree_attention(q.cuda(), pool.on_gpu(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  torch.zeros(batch + 1, dtype=torch.int32, device="cuda"), out=out)
        assert bool((out == 7.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_many_sequences_in_every_width(kind, dim):
    """2600 sequences, a few of which have tokens: more than a tile of them, one, none of their rows seen."""
    gen = torch.Generator().manual_seed(dim)
    kinds = kind.split("-")
    n = [0] * 2600
    n[0], n[3], n[700], n[701], n[2598], n[2599] = 3, 140, 1, 64, 70, 2
    lens = [3 * x // 2 + (x > 0) for x in n]
    lens[701] = 0
    table, pages = P.table_for(lens, 16, gen)
    pool = P.Pool(kinds[-1], pages, 16, 1, dim, "rows", gen)
    q = torch.randn(sum(n) + 3, 2, dim, generator=gen).to(P.DT[kinds[0]])
    say(f"[gpu] {kind} heads of {dim}")
    _tree(q, pool, table, lens, n, 16, max_len=max(lens))
    if len(kinds) == 1:
        k, v = (torch.randn(sum(n) + 3, 1, dim, generator=gen).to(q.dtype) for _ in range(2))
        for causal in (True, False):
            _prompt(q, k, v, n, causal=causal)


def test_eight_times_the_sequences_take_eight_times_as_long():
    """... and not the square of it (64 times): every workgroup finds its sequence among them in a few steps."""
    took = []
    for batch in (4096, 32768):
        q = torch.randn(batch, 8, 64, device="cuda").to(torch.bfloat16)
        starts = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
        out = torch.zeros_like(q)
        call = lambda: L.tc_prompt_attention(q, q, q, starts, out=out)
        call()
        torch.cuda.synchronize()
        best = 1e9
        for _ in range(5):
            t = time.perf_counter()
            call()
            torch.cuda.synchronize()
            best = min(best, time.perf_counter() - t)
        took.append(best)
        assert torch.equal(out, q)  # a token alone sees itself
    say(f"[gpu] {took[0] * 1e3:.2f} and {took[1] * 1e3:.2f} ms")
    assert took[1] < 24 * took[0]
