"""The paged key-value cache on the GPU: append, attention of one new token, eviction, and their run together,
against the definitions in 64 bits on the host."""

import math

import pytest
import torch

import layout_permuting_copy_amd as L
import paged_ref as R
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


def _same(got, want, what):
    """Equal bits; NaN codes of any kind are equal."""
    got = got.cpu()
    same = R.bits(got.contiguous()) == R.bits(want.contiguous())
    nan = got.float().isnan() & want.float().isnan()
    assert bool((same | nan).all()), f"{what}: {int((~(same | nan)).sum())} of {same.numel()} differ"


def _close(got, want, tol, what, out_dtype=None):
    got = got.cpu().double()
    if out_dtype is not None:  # out's own rounding
        tol = tol + torch.finfo(out_dtype).eps / 2 * (want.abs() + tol) + torch.finfo(out_dtype).smallest_normal * 2.0 ** -8
    nan = got.isnan() & want.isnan()
    fine = nan | (got == want) | ((got - want).abs() <= tol)
    if not bool(fine.all()):
        bad = torch.nonzero(~fine)[0].tolist()
        at = tuple(bad)
        raise AssertionError(f"{what}: {int((~fine).sum())} of {fine.numel()} off; at {at} got {got[at]} want {want[at]} "
                             f"tolerance {tol[at]}")


def _attend(q, pool, table, lens, page, weights=None, max_len=None, scale=None, check=True):
    """The call on the host's inputs, checked against the definition; returns (out, lse, weights)."""
    cache = pool.on_gpu()
    batch, heads = q.shape[0], pool.k.shape[2]
    most = max(max(lens), 1) if max_len is None else max_len
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    w = wo = None
    if weights is not None:
        w = weights.cuda()
        wo = w.clone()
    before = [x.clone() for x in R.cache_tensors(cache)]
    out = L.tc_paged_attention(q.cuda(), cache, table.cuda(), _i32(lens), scale=scale, max_len=most, lse=lse, weights=w,
                               weights_out=wo)
    torch.cuda.synchronize()
    for x, y in zip(before, R.cache_tensors(cache)):
        _same(y, x.cpu(), "the cache")
    if check:
        ref = R.attention(q, pool, table, [min(n, most) for n in lens], page, scale)
        _close(out, ref[0], ref[3], "out", q.dtype)
        _close(lse, ref[1], ref[4], "lse")
        if weights is not None:
            n = ref[2].shape[2]
            want = weights.double().clone()
            want[:, :, :n] += ref[2]
            tol = torch.zeros_like(want)
            tol[:, :, :n] = ref[5] + 2 * R.STEP32 * want[:, :, :n].abs()
            for b, m in enumerate(lens):
                tol[b, :, m:] = 0
            _close(wo, want, tol, "weights")
    return out, lse, wo


SHAPES = [  # heads, group, head_dim, page, order of the pool
    (1, 1, 16, 16, "rows"), (2, 1, 64, 16, "heads"), (2, 4, 128, 16, "rows"), (3, 5, 80, 24, "rows"),
    (1, 16, 256, 16, "heads"), (2, 17, 96, 1, "rows"), (1, 33, 128, 64, "pairs"), (5, 3, 48, 8, "heads"),
    (1, 40, 256, 32, "rows"), (2, 2, 192, 100, "pairs"), (8, 8, 128, 48, "heads"), (1, 12, 32, 7, "rows"),
]
LENS = [[1], [0, 1, 2, 15, 16, 17], [31, 0, 32, 33, 127, 128, 129], [257, 5, 511, 255, 256], [1300, 64, 1, 0, 2049]]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_attention(kind, shape):
    heads, group, dim, page, major = shape
    kinds = kind.split("-")
    for t, lens in enumerate(LENS):
        say(f"[gpu] attention {kind} {shape} lens={lens}")
        gen = torch.Generator().manual_seed(17 * t + dim)
        table, pages = R.table_for(lens, page, gen, junk=(1 << 30) if t % 2 else -5)
        pool = R.Pool(kinds[-1], pages, page, heads, dim, major, gen)
        q = (1.5 * torch.randn(len(lens), heads * group, dim, generator=gen)).to(R.DT[kinds[0]])
        w = torch.rand(len(lens), heads, max(max(lens), 1) + 3, generator=gen) if t % 2 == 0 else None
        _attend(q, pool, table, lens, page, w)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("page", [16, 24])
def test_attention_ignores_rows_past_the_end_and_missing_pages(kind, page):
    """Rows past a sequence's length hold NaN, pages that the table does not name hold NaN, and entries that name
    no page drop their rows; a sequence whose pages are all missing gives zeros."""
    gen = torch.Generator().manual_seed(3)
    lens = [70, 333, 16, 1, 48, 600]
    table, pages = R.table_for(lens, page, gen, spare=3, junk=2 ** 31 - 1)
    pool = R.Pool(kind, pages, page, 2, 64, "rows", gen)
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        i = torch.arange(n)
        used[table[b][i // page].long(), i % page] = True
    for x in pool.tensors():
        y = R.bits(x)
        y[~used] = R.bits(torch.full((1,), float("nan")).to(x.dtype))[0]
    q = torch.randn(len(lens), 6, 64, generator=gen).to(torch.float16 if kind == "fp16" else torch.bfloat16)
    say(f"[gpu] NaN past the end {kind} page={page}")
    _attend(q, pool, table, lens, page)
    table[1, 3] = -1
    table[1, 7] = pages
    table[5, 0] = -(2 ** 31)
    table[4, :] = pages + 5
    say(f"[gpu] missing pages {kind} page={page}")
    out, lse, _ = _attend(q, pool, table, lens, page, torch.zeros(len(lens), 2, 600))
    assert not out[4].any() and bool((lse[4] == -math.inf).all())


def test_attention_of_infinite_and_nan_values():
    """A NaN or infinite logit makes its head NaN, as exp(inf - inf) is; logits of -infinity weigh nothing, and a
    head with no others gives zeros; other heads and sequences keep their values."""
    gen = torch.Generator().manual_seed(4)
    lens, page = [40, 40, 40, 40, 300], 16
    table, pages = R.table_for(lens, page, gen)
    pool = R.Pool("bf16", pages, page, 2, 64, "rows", gen)
    q = torch.randn(5, 4, 64, generator=gen).abs().to(torch.bfloat16) + 0.5
    at = lambda b, i: (int(table[b, i // page]), i % page)
    pool.k[at(0, 7)][0, 5] = float("nan")
    pool.k[at(1, 20)][1, 5] = float("inf")
    pool.k[at(2, 39)][0, 5] = float("-inf")
    for i in range(40):
        pool.k[at(3, i)][1, 0] = float("-inf")
    pool.v[at(4, 299)][1, 3] = float("nan")
    for wide in (40, 300):
        n = [min(m, wide) for m in lens]
        say(f"[gpu] infinities, lengths {n}")
        out, lse, w = _attend(q, pool, table, n, page, torch.zeros(5, 2, 300))
        assert bool(out[0, :2].isnan().all()) and not bool(out[0, 2:].isnan().any())
        assert bool(out[1, 2:].isnan().all()) and not bool(out[1, :2].isnan().any())
        assert not bool(out[2].isnan().any()) and float(w[2, 0, 39]) == 0.0
        assert not out[3, 2:].any() and bool((lse[3, 2:] == -math.inf).all())


def test_attention_lowest_values_and_sharp_rows():
    """Keys of the type's lowest value (logits far below the others), one row that takes all the weight, equal rows."""
    gen = torch.Generator().manual_seed(5)
    lens, page = [100, 100, 100], 16
    table, pages = R.table_for(lens, page, gen)
    for kind in ("bf16", "fp16"):
        dt = R.DT[kind]
        pool = R.Pool(kind, pages, page, 1, 64, "rows", gen)
        q = torch.zeros(3, 2, 64).to(dt)
        q[:, :, 0] = 1.0
        for i in range(100):
            p, r = int(table[0, i // page]), i % page
            if i % 3:
                pool.k[p, r, 0, 0] = torch.finfo(dt).min / 4
        pool.k[int(table[1, 2]), 5, 0, 0] = 400.0
        pool.k[table[2][:7].long(), :, 0, :] = 0.0
        say(f"[gpu] lowest values {kind}")
        out, _, _ = _attend(q, pool, table, lens, page, scale=1.0)
        _same(out[1, 0], pool.v[int(table[1, 2]), 5, 0], "the row that takes all the weight")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_attention_of_many_light_rows_beside_a_heavy_one(kind):
    """One row whose weight is e^17.5 times that of each of 8000 others, which hold all of out."""
    gen = torch.Generator().manual_seed(14)
    lens, page = [8001] * 4, 16
    table, pages = R.table_for(lens, page, gen)
    pool = R.Pool(kind, pages, page, 1, 64, "rows", gen)
    pool.k.zero_()
    pool.v.fill_(1.0)
    for b in range(4):
        pool.k[int(table[b, 0]), b, 0, 0] = 17.5
        pool.v[int(table[b, 0]), b, 0] = 0.0
    q = torch.zeros(4, 2, 64).to(R.DT[kind])
    q[:, :, 0] = 1.0
    for most in (1000, 8001):
        say(f"[gpu] light rows {kind}, {most} rows")
        _attend(q, pool, table, [min(n, most) for n in lens], page, scale=1.0)


def test_attention_views_and_other_layouts():
    """q and out as slices, a table with strides, a strided lse, weights of one buffer grown in place, a small max_len."""
    gen = torch.Generator().manual_seed(6)
    lens, page, heads, group, dim = [200, 77, 300], 16, 2, 3, 64
    table, pages = R.table_for(lens, page, gen)
    pool = R.Pool("bf16", pages, page, heads, dim, "pairs", gen)
    qkv = torch.randn(3, 2 * heads * group + 5, dim + 3, generator=gen).to(torch.bfloat16)
    q = qkv[:, 1:1 + 2 * heads * group:2, 1:1 + dim]
    ref = R.attention(q, pool, table, lens, page)
    cache = pool.on_gpu()
    wide = torch.full((2 * table.shape[1], 3), -1, dtype=torch.int32)
    wide[::2] = table.t()
    lse = torch.zeros(heads * group, 5, device="cuda")
    out = torch.full((heads * group, 3, 2 * dim), 9.0, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(3, 400, heads, device="cuda")
    qg = qkv.cuda()[:, 1:1 + 2 * heads * group:2, 1:1 + dim]
    for k in range(3):
        L.tc_paged_attention(qg, cache, wide.cuda().t()[:, ::2], _i32(lens), out=out.transpose(0, 1)[..., 3:3 + dim],
                             lse=lse[:, 1:4].t(), weights=w.transpose(1, 2))
    torch.cuda.synchronize()
    _close(out.transpose(0, 1)[..., 3:3 + dim], ref[0], ref[3], "out", torch.bfloat16)
    _close(lse[:, 1:4].t(), ref[1], ref[4], "lse")
    assert bool((out[..., :3] == 9).all()) and bool((out[..., 3 + dim:] == 9).all()) and not lse[:, 0].any()
    want = torch.ones(3, heads, 400, dtype=torch.float64)
    want[:, :, :300] += 3 * ref[2]
    tol = torch.zeros_like(want)
    tol[:, :, :300] = 3 * ref[5] + 6 * R.STEP32 * want[:, :, :300] * (ref[2] > 0)
    _close(w.transpose(1, 2), want, tol, "weights")
    say("[gpu] max_len shorter than the lengths")
    _attend(q.contiguous(), pool, table, lens, page, torch.zeros(3, heads, 300), max_len=130)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_of_many_and_of_long_sequences(kind):
    """More sequences than lanes of a wave and than runs of rows; one sequence in more parts than lanes; one long
    sequence among short ones."""
    gen = torch.Generator().manual_seed(9)
    lengths = [[int(x) for x in torch.randint(0, 700, (300,), generator=gen)], [70003], [3, 1, 20011, 0, 90, 1],
               [513] * 70 + [0] * 70 + [1400]]
    for heads, page, lens in zip((1, 1, 2, 9), (16, 24, 32, 7), lengths):
        table, pages = R.table_for(lens, page, gen)
        pool = R.Pool(kind, pages, page, heads, 32, "heads", gen)
        q = torch.randn(len(lens), 2 * heads, 32, generator=gen).to(torch.bfloat16)
        say(f"[gpu] {len(lens)} sequences, longest {max(lens)}, {heads} heads, {kind}")
        _attend(q, pool, table, lens, page, torch.zeros(len(lens), heads, max(lens)) if len(lens) < 300 else None)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("page", [16, 12, 7])
@pytest.mark.parametrize("dim", [16, 80, 192])
def test_attention_reads_no_other_heads_rows(kind, page, dim):
    """Rows shorter than the kernel's lanes cover, beside a head whose rows are NaN, and at the very end of a pool."""
    gen = torch.Generator().manual_seed(12)
    lens = [45, 200]
    table, pages = R.table_for(lens, page, gen)
    pool = R.Pool(kind, pages, page, 3, dim, "rows", gen)
    for x in (pool.k, pool.v):
        R.bits(x)[:, :, 1] = R.bits(torch.full((1,), float("nan")).to(x.dtype))[0]
    q = torch.randn(2, 6, dim, generator=gen).to(torch.float16 if kind == "fp16" else torch.bfloat16)
    say(f"[gpu] NaN in a neighbouring head {kind} page={page} dim={dim}")
    out, _, _ = _attend(q, pool, table, lens, page, torch.zeros(2, 3, 200))
    assert bool(out[:, 2:4].isnan().all()) and not bool(out[:, :2].isnan().any()) and not bool(out[:, 4:].isnan().any())


@pytest.mark.parametrize("batch", [31, 33, 300])
def test_attention_around_the_uncut_lengths(batch):
    """Lengths up to 1024 with and without a sequence and head for every CU: uncut and cut calls."""
    gen = torch.Generator().manual_seed(13)
    lens = [int(x) for x in torch.randint(0, 1025, (batch,), generator=gen)]
    lens[1], lens[2] = 1024, 0
    heads = 8 if batch < 300 else 1
    table, pages = R.table_for(lens, 32, gen)
    pool = R.Pool("bf16", pages, 32, heads, 16, "rows", gen)
    q = torch.randn(batch, heads, 16, generator=gen).to(torch.bfloat16)
    for most in (1024, 1025):
        say(f"[gpu] {batch} sequences, max_len {most}")
        _attend(q, pool, table, lens, 32, max_len=most)


def test_attention_scales():
    gen = torch.Generator().manual_seed(10)
    lens, page = [40, 600], 16
    table, pages = R.table_for(lens, page, gen)
    pool = R.Pool("fp16", pages, page, 1, 64, "rows", gen)
    q = torch.randn(2, 3, 64, generator=gen).to(torch.float16)
    for scale in (-0.3, 0.0, 1.0, 3.0):
        say(f"[gpu] scale {scale}")
        _attend(q, pool, table, lens, page, scale=scale)


def test_calls_from_threads_on_separate_streams():
    import threading
    jobs, errors = [], []
    for i in range(6):
        gen = torch.Generator().manual_seed(90 + i)
        lens = [50 * i + 1, 900 - 100 * i, 17]
        table, pages = R.table_for(lens, 16, gen)
        pool = R.Pool(("bf16", "fp16", "e4m3")[i % 3], pages, 16, 2, 64, "rows", gen)
        q = torch.randn(3, 8, 64, generator=gen).to(torch.float16 if i % 3 == 1 else torch.bfloat16)
        ref = R.attention(q, pool, table, lens, 16)
        jobs.append((pool.on_gpu(), q.cuda(), table.cuda(), _i32(lens), ref))
    torch.cuda.synchronize()

    def work(cache, q, table, lens, ref):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(8):
                    w = torch.zeros(3, 2, 912, device="cuda")
                    out = L.tc_paged_attention(q, cache, table, lens, weights=w, max_len=912)
                    with pytest.raises(L.TileCopyError):
                        L.tc_paged_attention(q, cache, table, lens, max_len=-1)
                    s.synchronize()
                    _close(out, ref[0], ref[3], "out", q.dtype)
        except BaseException as e:  # reported below
            errors.append(repr(e))

    say(f"[gpu] {len(jobs)} threads")
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:2]


def test_attention_equal_calls_give_equal_bits():
    gen = torch.Generator().manual_seed(7)
    lens, page = [5000, 1234], 16
    table, pages = R.table_for(lens, page, gen)
    pool = R.Pool("bf16", pages, page, 2, 128, "rows", gen)
    q = torch.randn(2, 8, 128, generator=gen).to(torch.bfloat16)
    a = _attend(q, pool, table, lens, page, torch.zeros(2, 2, 5000))
    b = _attend(q, pool, table, lens, page, torch.zeros(2, 2, 5000), check=False)
    for x, y in zip(a, b):
        _same(x, y.cpu(), "a second call")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_far_into_a_large_pool(kind):
    """Pages beyond 2^32 bytes and 2^31 elements of the pool, a page stride of its own."""
    pages, page, heads, dim = 70000, 16, 8, 256
    dt = R.DT[kind]
    say(f"[gpu] a pool of {pages * page * heads * dim} elements a side")
    k = torch.empty(pages, page, heads, dim, dtype=dt, device="cuda")
    v = torch.empty(pages, page, heads, dim, dtype=dt, device="cuda")
    ks = vs = None
    if kind == "e4m3":
        ks, vs = (torch.empty(pages, page, heads, device="cuda") for _ in range(2))
    cache = L.PagedCache(k, v, ks, vs)
    gen = torch.Generator().manual_seed(8)
    n = 150
    names = torch.tensor([[69999, 0, 65537, 69998, 33000, 68000, 1, 66000, 69000, 69001]], dtype=torch.int32)
    new_k, new_v = (torch.randn(n, heads, dim, generator=gen).to(torch.bfloat16) for _ in range(2))
    L.tc_paged_append(cache, new_k.cuda(), new_v.cuda(), names.cuda(), _i32([n]), token_starts=_i32([0, n]))
    small = R.Pool("bf16" if kind != "e4m3" else kind, 10, page, heads, dim, "rows", gen)
    for i in range(n):
        for dst, sc, new in ((small.k, small.ks, new_k), (small.v, small.vs, new_v)):
            if kind == "e4m3":
                c, s = R.quantise(new[i])
                R.bits(dst)[i // page, i % page] = R.bits(c)
                sc[i // page, i % page] = s
            else:
                dst[i // page, i % page] = new[i]
    near = torch.arange(10, dtype=torch.int32).view(1, 10)
    q = torch.randn(1, heads * 2, dim, generator=gen).to(torch.bfloat16)
    lse = torch.empty(1, heads * 2, device="cuda")
    out = L.tc_paged_attention(q.cuda(), cache, names.cuda(), _i32([n]), lse=lse)
    ref = R.attention(q, small, near, [n], page)
    _close(out, ref[0], ref[3], "out", q.dtype)
    _close(lse, ref[1], ref[4], "lse")
    # and an eviction out of it
    into = R.Pool(kind, 5, page, heads, dim, "rows", fill=0.0).on_gpu()
    w = torch.rand(1, heads, n, generator=gen)
    names_to = torch.tensor([[4, 2, 0, 1]], dtype=torch.int32)
    _, kept = L.tc_paged_evict(cache, names.cuda(), _i32([n]), w.cuda(), into, names_to.cuda(), 64, 8, max_len=n)
    kept = kept.cpu()
    for h in range(heads):
        rows = R.keep_rows(w[0, h].tolist(), n, 64, 8)
        assert kept[0, h].tolist() == rows
        for j in (0, 31, 63):
            _same(into.k[int(names_to[0, j // page]), j % page, h], small.k[rows[j] // page, rows[j] % page, h], "key row")
            _same(into.v[int(names_to[0, j // page]), j % page, h], small.v[rows[j] // page, rows[j] % page, h], "value row")


# ---- append ----------------------------------------------------------------------------------

def _append_ref(pool, k, v, table, lens, starts, page):
    for b in range(len(lens)):
        first, end = (b, b + 1) if starts is None else (starts[b], starts[b + 1])
        for t in range(first, end):
            i = lens[b] - (end - t)
            if i < 0 or i // page >= table.shape[1]:
                continue
            p = int(table[b, i // page])
            if not 0 <= p < pool.k.shape[0]:
                continue
            for dst, sc, new in ((pool.k, pool.ks, k), (pool.v, pool.vs, v)):
                if sc is None:
                    dst[p, i % page] = new[t]
                else:
                    c, s = R.quantise(new[t])
                    R.bits(dst)[p, i % page] = R.bits(c)
                    sc[p, i % page] = s


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"])
@pytest.mark.parametrize("shape", [(1, 16, 16, "rows"), (8, 128, 16, "heads"), (3, 80, 5, "rows"), (2, 256, 64, "pairs"),
                                   (5, 32, 1, "rows"), (2, 48, 24, "pairs"), (7, 64, 100, "heads")],
                         ids=lambda s: "x".join(map(str, s)))
def test_append(kind, shape):
    """Single tokens and chunks of unequal lengths, empty ones and padding among them, from aligned and
    unaligned rows; every byte that is not a new row's stays as it was."""
    heads, dim, page, major = shape
    kinds = kind.split("-")
    for t, (chunks, past, pad) in enumerate([([1] * 5, [0, 3, 99, 1, 17], 0), ([3, 0, 130, 1, 0, 65], [0, 9, 15, 16, 0, 1], 9),
                                             ([1, 2, 0] * 30, [1] * 90, 2), ([7], [0], 0)]):
        gen = torch.Generator().manual_seed(40 + t)
        lens = [a + b for a, b in zip(chunks, past)]
        table, pages = R.table_for(lens, page, gen, spare=2, junk=-1)
        if t == 1:
            table[5, (lens[5] - 1) // page] = pages  # no page: those rows go nowhere
        pool = R.Pool(kinds[-1], pages, page, heads, dim, major, gen)
        tokens = sum(chunks) + pad
        off = 1 if t % 2 else 0
        rows = torch.randn(tokens, 3 * heads, dim + 8 * off, generator=gen).to(R.DT[kinds[0]])
        rows[0, :, ::3] *= 37.0
        if tokens > 2:
            rows[2] = 0.0
        starts = None if t == 0 else [sum(chunks[:i]) for i in range(len(chunks) + 1)]
        cut = lambda x, i: x[:, i * heads:(i + 1) * heads, off:off + dim]
        cache = pool.on_gpu()
        w = torch.ones(len(lens), heads, 64, device="cuda")
        say(f"[gpu] append {kind} {shape} chunks={chunks[:8]}")
        g = rows.cuda()
        L.tc_paged_append(cache, cut(g, 1), cut(g, 2), table.cuda(), _i32(lens), weights=w,
                          token_starts=None if starts is None else _i32(starts))
        torch.cuda.synchronize()
        _append_ref(pool, cut(rows, 1), cut(rows, 2), table, lens, starts, page)
        for x, y, name in zip(R.cache_tensors(cache), pool.tensors(), ("keys", "values", "key scales", "value scales")):
            _same(x, y, name)
        for b, n in enumerate(lens):
            z = torch.ones(64)
            for i in range(n - chunks[b], min(n, 64)):
                if 0 <= int(table[b, i // page]) < pages:
                    z[i] = 0.0
            assert torch.equal(w[b].cpu(), z.expand(heads, 64)), (b, n)


def test_append_8bit_scales_at_the_edges():
    """Rows of zeros, of the smallest and largest values, with infinities and NaN: scale and codes as defined."""
    for name in ("bf16", "fp16"):
        dt = R.DT[name]
        f = torch.finfo(dt)
        gen = torch.Generator().manual_seed(50)
        rows = torch.randn(64, 1, 32, generator=gen).to(dt)
        rows[0] = 0.0
        rows[1] = f.max
        rows[2] = f.smallest_normal * (torch.rand(1, 32, generator=gen).to(dt) - 0.5)
        rows[3, 0, 4] = float("inf")
        rows[4, 0, 31] = float("nan")
        rows[5, 0, 0] = float("-inf")
        rows[6, 0, 3] = f.max
        rows[7] = f.tiny / 2
        rows[8:40] = (rows[8:40].float() * torch.exp2(torch.linspace(-130 if name == "bf16" else -20, 10, 32)).view(32, 1, 1)).to(dt)
        pool = R.Pool("e4m3", 4, 16, 1, 32, "rows", fill=1.0)
        cache = pool.on_gpu()
        table = torch.arange(4, dtype=torch.int32).view(1, 4)
        say(f"[gpu] 8-bit edges {name}")
        L.tc_paged_append(cache, rows.cuda(), rows.cuda(), table.cuda(), _i32([64]), token_starts=_i32([0, 64]))
        _append_ref(pool, rows, rows, table, [64], [0, 64], 16)
        for x, y, what in zip(R.cache_tensors(cache), pool.tensors(), ("keys", "values", "key scales", "value scales")):
            _same(x, y, what)


# ---- eviction --------------------------------------------------------------------------------

def _evict_check(pool, table, lens, page, w, into, into_table, into_page, budget, recent, max_len=None, same_pool=False):
    heads = pool.k.shape[2]
    src = pool.on_gpu()
    dst = src if same_pool else into.on_gpu()
    most = max(1, min(budget, max(max(lens), 1) if max_len is None else max_len))
    wo = torch.full((len(lens), heads, most + 2), -3.0, device="cuda")
    kept = torch.full((len(lens), heads, most + 1), 77, dtype=torch.int32, device="cuda")
    lens_out, _ = L.tc_paged_evict(src, table.cuda(), _i32(lens), w.cuda(), dst, into_table.cuda(), budget, recent,
                                   max_len=max(max(lens), 1) if max_len is None else max_len, weights_out=wo, kept=kept)
    torch.cuda.synchronize()
    ref = pool if same_pool else into
    taken = [x.clone() for x in pool.tensors()]
    want_kept = torch.full(kept.shape, -1, dtype=torch.int32)
    want_w = torch.full(wo.shape, -3.0)
    for b, n in enumerate(lens):
        n = n if max_len is None else min(n, max_len)
        assert int(lens_out[b]) == min(n, budget)
        for h in range(heads):
            rows = R.keep_rows(w[b, h].tolist(), n, budget, recent)
            want_kept[b, h, :len(rows)] = torch.tensor(rows, dtype=torch.int32)
            if not rows:
                continue
            i, j = torch.tensor(rows), torch.arange(len(rows))
            want_w[b, h, :len(rows)] = w[b, h, i]
            sp, dp = table[b][i // page].long(), into_table[b][j // into_page].long()
            ok = (sp >= 0) & (sp < pool.k.shape[0]) & (dp >= 0) & (dp < ref.k.shape[0])
            i, j, sp, dp = i[ok], j[ok], sp[ok], dp[ok]
            for x, y in zip(taken, ref.tensors()):
                R.bits(y)[dp, j % into_page, h] = R.bits(x)[sp, i % page, h]
    assert torch.equal(kept.cpu(), want_kept)
    _same(wo, want_w, "weights")
    for x, y in zip(R.cache_tensors(dst), ref.tensors()):
        _same(x, y, "dst")
    if not same_pool:
        for x, y in zip(R.cache_tensors(src), pool.tensors()):
            _same(x, y, "src")


def _weights(batch, heads, cap, gen):
    """Heavy tails, zeros of both signs, ties, negative values and NaN among them."""
    w = torch.exp(2 * torch.randn(batch, heads, cap, generator=gen))
    u = torch.rand(w.shape, generator=gen)
    w = torch.where(u < 0.3, torch.floor(w * 4) / 4, w)
    w = torch.where((u > 0.3) & (u < 0.35), -torch.zeros_like(w), w)
    w = torch.where((u > 0.35) & (u < 0.4), -w, w)
    return torch.where(u > 0.995, torch.full_like(w, float("nan")), w)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("shape", [(1, 16, 16, 16, "rows"), (3, 128, 16, 24, "heads"), (2, 80, 7, 16, "rows"), (2, 256, 64, 1, "pairs"),
                                   (4, 64, 100, 32, "heads")], ids=lambda s: "x".join(map(str, s)))
def test_evict(kind, shape):
    heads, dim, page, into_page, major = shape
    for t, (lens, budget, recent) in enumerate([([1, 0, 5, 40, 41], 40, 8), ([300, 64, 65, 1100, 63], 64, 0), ([130, 64, 200], 64, 64),
                                                ([2500, 1030, 1024, 17], 1000, 31), ([77, 3], 1, 0), ([50], 1, 1), ([64, 9], 200, 5)]):
        gen = torch.Generator().manual_seed(60 + t)
        table, pages = R.table_for(lens, page, gen)
        into_table, into_pages = R.table_for([min(n, budget) for n in lens], into_page, gen,
                                             cols=(min(budget, max(lens)) + into_page - 1) // into_page)
        pool = R.Pool(kind, pages, page, heads, dim, major, gen)
        into = R.Pool(kind, into_pages, into_page, heads, dim, "rows" if t % 2 else "pairs", fill=0.0)
        say(f"[gpu] evict {kind} {shape} lens={lens} budget={budget} recent={recent}")
        _evict_check(pool, table, lens, page, _weights(len(lens), heads, max(lens) + t, gen), into, into_table, into_page, budget,
                     recent)


def test_evict_equal_weights_keep_the_lowest_rows():
    gen = torch.Generator().manual_seed(70)
    for lens, budget, recent in (([5000, 1500], 700, 100), ([1025, 2900], 1024, 0)):
        table, pages = R.table_for(lens, 16, gen)
        into_table, into_pages = R.table_for([budget] * 2, 16, gen)
        for value in (0.0, 1.5, float("nan"), -2.0, float("inf")):
            pool = R.Pool("bf16", pages, 16, 1, 16, "rows", gen)
            into = R.Pool("bf16", into_pages, 16, 1, 16, "rows", fill=0.0)
            w = torch.full((2, 1, max(lens)), value)
            say(f"[gpu] equal weights {value}")
            _evict_check(pool, table, lens, 16, w, into, into_table, 16, budget, recent)


def test_evict_of_infinite_weights_into_strided_rows():
    """Weights of both infinities, zeros of both signs and the lowest and highest numbers; kept and weights_out with
    strides between their columns give what dense ones do."""
    gen = torch.Generator().manual_seed(15)
    page, heads = 16, 2
    for lens, budget, recent in (([700, 90], 64, 7), ([3000, 1], 900, 0), ([40000, 20000], 5000, 100)):
        table, pages = R.table_for(lens, page, gen)
        into_table, into_pages = R.table_for([min(n, budget) for n in lens], page, gen)
        pool = R.Pool("bf16", pages, page, heads, 16, "rows", gen)
        into = R.Pool("bf16", into_pages, page, heads, 16, "rows", fill=0.0)
        w = torch.randn(2, heads, max(lens), generator=gen)
        pick = torch.randint(0, 40, w.shape, generator=gen)
        for i, x in enumerate((math.inf, -math.inf, 0.0, -0.0, 3.4e38, -3.4e38, 1e-42, -1e-42)):
            w[pick == i] = x
        w[1, 1] = -math.inf
        say(f"[gpu] infinite weights lens={lens}")
        _evict_check(pool, table, lens, page, w, into, into_table, page, budget, recent)
        got = []
        for step in (1, 3):
            kept = torch.full((2, heads, budget, step), 5, dtype=torch.int32, device="cuda")
            wo = torch.full((2, heads, budget, step), 5.0, device="cuda")
            L.tc_paged_evict(pool.on_gpu(), table.cuda(), _i32(lens), w.cuda(), into.on_gpu(), into_table.cuda(), budget, recent,
                             max_len=max(lens), weights_out=wo[..., 0], kept=kept[..., 0])
            torch.cuda.synchronize()
            assert bool((kept[..., 1:] == 5).all()) and bool((wo[..., 1:] == 5).all())
            got.append((kept[..., 0].cpu(), wo[..., 0].cpu()))
        assert torch.equal(got[0][0], got[1][0])
        _same(got[1][1], got[0][1], "weights")


def test_evict_long_rows_in_one_pool_and_missing_pages():
    """Into other pages of the same pool; pages missing on either side; a max_len under the lengths; a long sequence."""
    gen = torch.Generator().manual_seed(71)
    lens, budget, recent, page = [70001, 900], 500, 50, 16
    both, pages = R.table_for(lens + [500, 500], page, gen)
    table, into_table = both[:2].contiguous(), both[2:, :32].contiguous()
    pool = R.Pool("bf16", pages, page, 1, 32, "rows", gen)
    table[1, 4] = -1
    into_table[0, 3] = pages + 1
    w = _weights(2, 1, 70001, gen)
    say("[gpu] evict within one pool")
    _evict_check(pool, table, lens, page, w, None, into_table, page, budget, recent, same_pool=True)
    say("[gpu] evict from 20001 rows")
    _evict_check(pool, table, lens, page, w, R.Pool("bf16", pages, page, 1, 32, "rows", fill=0.0), into_table, page, budget, recent,
                 max_len=20001)
    say("[gpu] evict with a max_len under the lengths")
    _evict_check(pool, table, lens, page, w, R.Pool("bf16", pages, page, 1, 32, "heads", fill=0.0), into_table, page, budget,
                 recent, max_len=801)


# ---- together --------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3"])
def test_decoding_under_a_budget(kind):
    """Prompts appended, then steps of append and attention that add the weights up, the cache shrunk to its budget
    whenever a sequence outgrows it by a page: every step's outputs against the definition on the cache as it stands."""
    kinds = kind.split("-")
    heads, group, dim, page, budget, recent, slack = 2, 4, 64, 16, 96, 16, 16
    gen = torch.Generator().manual_seed(80)
    lens = [130, 40, 96, 1]
    batch, cap = len(lens), 160
    cols = cap // page
    pages = 2 * batch * cols
    pool = R.Pool(kinds[-1], pages, page, heads, dim, "heads", fill=0.0)
    cache = pool.on_gpu()
    order = torch.randperm(pages, generator=gen).to(torch.int32).view(2, batch, cols)
    side = 0
    table = order[0]
    w = torch.full((batch, heads, cap), 5.0, device="cuda")
    new = lambda n: torch.randn(n, heads, dim, generator=gen).to(R.DT[kinds[0]])
    starts = [sum(lens[:i]) for i in range(batch + 1)]
    k, v = new(sum(lens)), new(sum(lens))
    L.tc_paged_append(cache, k.cuda(), v.cuda(), table.cuda(), _i32(lens), token_starts=_i32(starts), weights=w)
    _append_ref(pool, k, v, table, lens, starts, page)
    evictions = 0
    for step in range(40):
        lens = [n + 1 for n in lens]
        k, v = new(batch), new(batch)
        L.tc_paged_append(cache, k.cuda(), v.cuda(), table.cuda(), _i32(lens), weights=w)
        _append_ref(pool, k, v, table, lens, None, page)
        q = torch.randn(batch, heads * group, dim, generator=gen).to(R.DT[kinds[0]])
        before = w.cpu().double()
        lse = torch.empty(batch, heads * group, device="cuda")
        out = L.tc_paged_attention(q.cuda(), cache, table.cuda(), _i32(lens), lse=lse, weights=w)
        ref = R.attention(q, pool, table, lens, page)
        n = ref[2].shape[2]
        _close(out, ref[0], ref[3], f"step {step} out", q.dtype)
        _close(lse, ref[1], ref[4], f"step {step} lse")
        _close(w[:, :, :n], before[:, :, :n] + ref[2], ref[5] + 2 * R.STEP32 * (before[:, :, :n] + ref[2]), f"step {step} weights")
        if max(lens) >= budget + slack:
            evictions += 1
            side ^= 1
            after = torch.full_like(w, -1.0)
            lens_out, kept = L.tc_paged_evict(cache, table.cuda(), _i32(lens), w, cache, order[side].cuda(), budget, recent,
                                              weights_out=after)
            host = w.cpu()
            taken = [x.clone() for x in pool.tensors()]
            for b, m in enumerate(lens):
                for h in range(heads):
                    rows = R.keep_rows(host[b, h].tolist(), m, budget, recent)
                    assert kept[b, h, :len(rows)].tolist() == rows
                    for j, i in enumerate(rows):
                        for x, y in zip(taken, pool.tensors()):
                            R.bits(y)[int(order[side][b, j // page]), j % page, h] = R.bits(x)[int(table[b, i // page]), i % page, h]
            lens, table, w = lens_out.tolist(), order[side], after
    assert evictions >= 2
    for x, y in zip(R.cache_tensors(cache), pool.tensors()):
        _same(x, y, "the pool at the end")


def test_a_captured_step_replays_with_new_contents():
    """Append and attention captured once and replayed while lengths, tables, tokens and the pool move on, with the
    program's own work between the replays; then two captured graphs side by side on two streams."""
    gen = torch.Generator().manual_seed(81)
    heads, group, dim, page, batch, cols = 2, 4, 128, 16, 3, 40
    pages = batch * cols
    pool = R.Pool("bf16", pages, page, heads, dim, "rows", gen)
    cache = pool.on_gpu()
    table = torch.randperm(pages, generator=gen).to(torch.int32).view(batch, cols)
    t_d, lens_d = table.cuda(), _i32([1] * batch)
    q_d = torch.zeros(batch, heads * group, dim, device="cuda", dtype=torch.bfloat16)
    k_d, v_d = (torch.zeros(batch, heads, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.zeros(batch, heads, cols * page, device="cuda")
    wo = torch.zeros_like(w)
    graphs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        lse = torch.zeros(batch, heads * group, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            L.tc_paged_attention(q_d, cache, t_d, lens_d, lse=lse, weights=w, weights_out=wo)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            if not graphs:
                L.tc_paged_append(cache, k_d, v_d, t_d, lens_d)
            out = L.tc_paged_attention(q_d, cache, t_d, lens_d, lse=lse, weights=w, weights_out=wo if not graphs else w.clone())
        graphs.append((g, out, lse, s))
    for step, lens in enumerate([[5, 300, 1], [6, 301, 640], [7, 0, 2], [639, 16, 17], [1, 1, 1]]):
        say(f"[gpu] replay {step}")
        q = torch.randn(batch, heads * group, dim, generator=gen).to(torch.bfloat16)
        k, v = (torch.randn(batch, heads, dim, generator=gen).to(torch.bfloat16) for _ in range(2))
        q_d.copy_(q), k_d.copy_(k), v_d.copy_(v), lens_d.copy_(_i32(lens))
        (torch.randn(1 << 20, device="cuda") * 2).sum().item()
        _append_ref(pool, k, v, table, lens, None, page)
        graphs[0][0].replay()
        torch.cuda.synchronize()
        for g, _, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        ref = R.attention(q, pool, table, lens, page)
        n = ref[2].shape[2]
        for g, out, lse, _ in graphs:
            _close(out, ref[0], ref[3], "out", q.dtype)
            _close(lse, ref[1], ref[4], "lse")
        for b, m in enumerate(lens):
            _close(wo[b, :, :m], ref[2][b, :, :m], ref[5][b, :, :m] + 2 * R.STEP32 * ref[2][b, :, :m], "weights")


def test_calls_on_another_stream():
    """The stream argument, as an object and as a handle: work and memory of the call belong to that stream."""
    gen = torch.Generator().manual_seed(82)
    lens, page = [700, 333], 16
    table, pages = R.table_for(lens, page, gen)
    pool = R.Pool("fp16", pages, page, 2, 64, "rows", gen)
    cache = pool.on_gpu()
    q = torch.randn(2, 6, 64, generator=gen).to(torch.float16)
    ref = R.attention(q, pool, table, lens, page)
    qd, td, ld = q.cuda(), table.cuda(), _i32(lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for stream in (s, s.cuda_stream, None):
        for _ in range(5):
            outs.append(L.tc_paged_attention(qd, cache, td, ld, stream=stream))
            torch.empty(1 << 16, device="cuda").fill_(float("nan"))  # memory the current stream may hand out again
    torch.cuda.synchronize()
    for out in outs:
        _close(out, ref[0], ref[3], "out", q.dtype)


def test_empty_calls():
    """No sequences, no tokens, no rows: nothing is written and nothing fails."""
    pool = R.Pool("bf16", 4, 16, 2, 64, "rows", fill=1.0)
    cache = pool.on_gpu()
    e = lambda *s, **k: torch.empty(*s, device="cuda", **k)
    i0 = e(0, dtype=torch.int32)
    L.tc_paged_append(cache, e(0, 2, 64, dtype=torch.bfloat16), e(0, 2, 64, dtype=torch.bfloat16), e(0, 3, dtype=torch.int32), i0)
    L.tc_paged_append(cache, e(0, 2, 64, dtype=torch.bfloat16), e(0, 2, 64, dtype=torch.bfloat16), _i32([[0], [1]]), _i32([3, 4]),
                      token_starts=_i32([0, 0, 0]))
    out = L.tc_paged_attention(e(0, 4, 64, dtype=torch.bfloat16), cache, e(0, 3, dtype=torch.int32), i0)
    assert out.shape == (0, 4, 64)
    for table, lens in ((_i32([[0], [1]]), _i32([0, -4])), (e(2, 0, dtype=torch.int32), _i32([3, 1]))):
        lse = torch.ones(2, 4, device="cuda")
        out = L.tc_paged_attention(torch.ones(2, 4, 64, device="cuda", dtype=torch.bfloat16), cache, table, lens, lse=lse)
        assert not out.any() and bool((lse == -math.inf).all())
    n, kept = L.tc_paged_evict(cache, _i32([[0], [1]]), _i32([0, -1]), torch.ones(2, 2, 16, device="cuda"), cache, _i32([[2], [3]]), 4)
    assert n.tolist() == [0, 0] and bool((kept == -1).all())
    L.tc_paged_evict(cache, e(0, 2, dtype=torch.int32), i0, e(0, 2, 32), cache, e(0, 2, dtype=torch.int32), 4)
    for x, y in zip(R.cache_tensors(cache), pool.tensors()):
        _same(x, y, "the cache")
    none = L.PagedCache(e(0, 16, 2, 64, dtype=torch.bfloat16), e(0, 16, 2, 64, dtype=torch.bfloat16))
    one = torch.ones(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    for cols in (1, 100):
        out = L.tc_paged_attention(one, none, torch.zeros(2, cols, device="cuda", dtype=torch.int32), _i32([16, 9]))
        assert not out.any()
        L.tc_paged_append(none, one[:, :2], one[:, :2], torch.zeros(2, cols, device="cuda", dtype=torch.int32), _i32([16, 9]))
