"""Attention over a paged cache at the edges of its number types, against values known in closed form or summed in 64 bits."""

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


def _half_step(dt, want, off):
    """How far rounding to dt takes a value that is within `off` of want: half a step, of subnormal numbers at least."""
    f = torch.finfo(dt)
    return f.eps / 2 * (want.abs() + off).clamp_min(f.smallest_normal)


def _one_sequence(k, v, q, page=16):
    """A cache of one head that holds k, v (rows, dim) as one sequence, and the call's other arguments."""
    n, dim = k.shape
    pages = (n + page - 1) // page
    pool_k, pool_v = (torch.zeros(pages, page, 1, dim, dtype=k.dtype) for _ in range(2))
    pool_k.view(-1, dim)[:n], pool_v.view(-1, dim)[:n] = k, v
    cache = L.PagedCache(pool_k.cuda(), pool_v.cuda())
    return q.view(1, -1, dim).cuda(), cache, torch.arange(pages, dtype=torch.int32).view(1, -1).cuda(), _i32([n])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("rows", [9, 300, 5000])
def test_attention_of_logits_far_from_zero(kind, sign, rows):
    """Logits of 2^21 to 2^30 on either side of zero: one row above all others has all the weight, the greatest ones of
    `equal` rows share it.  The others lie far more than the range of exp below, so p is 1 / equal for the greatest and 0
    for the rest, whatever the logits' own rounding; out is the mean of their values."""
    dt, dim, group = R.DT[kind], 32, 3
    gen = torch.Generator().manual_seed(rows)
    for power in (21, 23, 24, 25, 27, 29, 30):
        for equal in (1, 4):
            top = torch.randperm(rows, generator=gen)[:equal]
            # q k = 2^15 2^(power - 15) at the top, and below it 5 % down (sign 1) or up (-1) in magnitude
            near, far = 2.0 ** (power - 15), 2.0 ** (power - 15) * (0.95 if sign > 0 else 1.05)
            k = torch.zeros(rows, dim)
            k[:, 0] = sign * far
            k[top, 0] = sign * near
            v = torch.randn(rows, dim, generator=gen)
            q = torch.zeros(group, dim)
            q[:, 0] = 2.0 ** 15
            k, v, q = k.to(dt), v.to(dt), q.to(dt)
            say(f"[gpu] {kind} logits of {sign} * 2^{power}, {equal} of {rows} rows at the top")
            lse = torch.zeros(1, group, device="cuda")
            w = torch.zeros(1, 1, rows, device="cuda")
            out = L.tc_paged_attention(*_one_sequence(k, v, q), scale=1.0, max_len=rows, lse=lse, weights=w)
            want = v[top].double().mean(0)
            # the weights of 1 / equal are exact, their sum over the group too; the values' sum and its division are off by
            # half a step of fp32 each a term, out by half a step of its type
            tol = 2 * (equal + 2) * R.STEP32 * v[top].double().abs().max()
            tol = tol + _half_step(dt, want, tol)
            got = out[0].cpu().double()
            assert bool(((got - want).abs() <= tol).all()), (got[0], want)
            weight = torch.zeros(rows)
            weight[top] = group / equal
            assert torch.equal(w[0, 0].cpu(), weight), (w[0, 0].cpu()[top], group / equal)
            # lse: the logit times log2 e and back, each factor and product off by half a step of fp32
            x = sign * 2.0 ** power + math.log(equal)
            assert bool(((lse.cpu().double() - x).abs() <= 6 * R.STEP32 * abs(x)).all()), (lse, x)


def _two_parts(e):
    """e as the sum of two bf16 values, its rounding and the rest's."""
    hi = e.to(torch.float32).to(torch.bfloat16).double()
    return hi + (e - hi).to(torch.float32).to(torch.bfloat16).double()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"])
@pytest.mark.parametrize("group", [1, 20])
def test_attention_weights_have_the_precision_of_fp32(kind, group):
    """A row whose weight two bf16 values hold worst, and three rows of weight e^0 that cancel it down to less than 2^-10:
    out is then as far off as its weights and sums are.

    With e = 2^-24 and mag = sum p |v|: a logit of at most 1/4 is off by e / 2, its base-2 exponential by 2 e of its own, and
    a scale of the values adds e: 4 e of the row's weight, which holds half of mag.  The row enters the sums in at most three
    parts, the others (weight 1) in one: 6 additions of partial sums under half of mag, off by 2 e each where the matrix unit
    truncates.  The division is off by 2 e of out, which is small.  2 + 6 = 8 e of mag, and 12 with what those round to.  Two
    bf16 values leave 2^-17.7 of the row's weight, 39 e of mag."""
    kinds = kind.split("-")
    dt, kv, dim, page, main, fix = R.DT[kinds[0]], kinds[-1], 64, 16, 1, 3
    gen = torch.Generator().manual_seed(21)
    x = -torch.arange(1, 257, dtype=torch.float64) / 1024.0
    e = torch.exp(x)
    lost = (e - _two_parts(e)) / e
    worst = torch.argsort(lost, descending=True)[:main]
    x = torch.cat([x[worst], torch.zeros(fix, dtype=torch.float64)])
    e = torch.exp(x)
    n = main + fix
    pool = R.Pool(kv, 1, page, 1, dim, "rows", fill=0.0)
    if kv == "e4m3":
        pool.k[0, :n, 0, 0] = torch.tensor(-1.0).to(pool.k.dtype)
        pool.ks.fill_(0.0)
        pool.ks[0, :n, 0] = -x.float()
        pool.vs.fill_(1.0)
    else:
        pool.k[0, :n, 0, 0] = x.to(pool.k.dtype)
    v = torch.zeros(n, dim, dtype=torch.float64)
    to = lambda y: y.float().to(pool.v.dtype).float().double()
    v[:main] = to(16.0 + 8.0 * torch.rand(main, dim, generator=gen).double())
    for i in range(main, n):
        v[i] = to(-(e[:i, None] * v[:i]).sum(0))
    pool.v[0, :n, 0] = v.float().to(pool.v.dtype)
    p = e / e.sum()
    want, mag = p @ v, p @ v.abs()
    assert bool((want.abs() <= mag * 2.0 ** -10).all())
    q = torch.zeros(1, group, dim)
    q[..., 0] = 1.0
    say(f"[gpu] weights of {kind}, group {group}")
    out = L.tc_paged_attention(q.to(dt).cuda(), pool.on_gpu(), _i32([[0]]), _i32([n]), scale=1.0)
    off = (out[0].cpu().double() - want).abs()
    tol = 12 * R.STEP32 * mag + _half_step(dt, want, 12 * R.STEP32 * mag)
    say(f"[gpu] off by at most 2^{math.log2(float((off / mag).max()) + 1e-30):.2f} of the sum of magnitudes")
    assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("length", [-(2 ** 31), -(2 ** 31) + 2, -1, 0])
def test_append_to_a_sequence_of_negative_length_writes_nothing(length):
    """Lengths are taken as at least 0, also where the table holds 2^31 rows and more."""
    page = 1 << 20
    k, v = (torch.full((1, page, 1, 16), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = L.PagedCache(k, v)
    table = torch.zeros(1, 2 ** 31 // page, dtype=torch.int32, device="cuda")
    new = torch.ones(4, 1, 16, dtype=torch.bfloat16, device="cuda")
    say(f"[gpu] append to length {length}")
    L.tc_paged_append(cache, new[:1], new[:1], table, _i32([length]))
    L.tc_paged_append(cache, new, new, table, _i32([length]), token_starts=_i32([0, 4]))
    torch.cuda.synchronize()
    assert bool((k == 5.0).all()) and bool((v == 5.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 100, 5000])
@pytest.mark.parametrize("least", [0.25, 1.0])
def test_attention_beside_rows_of_the_lowest_value(kind, rows, least):
    """Two rows of three have the type's lowest key (or a quarter of it) and weigh nothing; the others are as exact as if
    they were alone.  With e = 2^-24: a logit x (one key element, so without a sum) is off by e |x| for each of scale and product, and
    by e for the difference to the maximum; a weight by twice that and 16 e for its exponential, the parts' factors and the
    division; a sum over rows is formed in n / 16 + 96 additions."""
    dt, dim, group = R.DT[kind], 64, 5
    gen = torch.Generator().manual_seed(rows)
    live = torch.arange(rows) % 3 == 0
    x = torch.randn(rows, generator=gen).to(dt)
    k = torch.zeros(rows, dim, dtype=dt)
    k[:, 0] = torch.where(live, x, torch.full((rows,), torch.finfo(dt).min).to(dt) * least)
    v = torch.randn(rows, dim, generator=gen).to(dt)
    v[~live] *= 64.0
    q = torch.zeros(group, dim, dtype=dt)
    q[:, 0] = 1.0 / 8.0  # (the lowest bf16 times log2 e would leave fp32's range)
    xs = x[live].double()
    p = torch.softmax(xs, 0)
    want, mag = p @ v[live].double(), p @ v[live].double().abs()
    dx = (3 * float(xs.abs().max()) + 1) * R.STEP32
    rel = 2 * dx + 16 * R.STEP32 + (rows / 16 + 96) * R.STEP32
    assert rel < 2.0 ** -14
    say(f"[gpu] {kind}, {rows} rows, lowest keys times {least}")
    lse, w = torch.zeros(1, group, device="cuda"), torch.zeros(1, 1, rows, device="cuda")
    out = L.tc_paged_attention(*_one_sequence(k, v, q), scale=8.0, max_len=rows, lse=lse, weights=w)
    assert bool(((out[0].cpu().double() - want).abs() <= rel * mag + _half_step(dt, want, rel * mag)).all())
    total = torch.logsumexp(xs, 0)
    assert bool(((lse.cpu().double() - total).abs() <= rel + 4 * R.STEP32 * (abs(total) + xs.abs().max())).all())
    weight = torch.zeros(rows, dtype=torch.float64)
    weight[live] = group * p
    assert bool(((w[0, 0].cpu().double() - weight).abs() <= (rel + group * R.STEP32) * weight).all())


def test_weights_and_sums_of_calls_from_threads():
    """Threads on streams of their own that add weights up: weights, log-sums and outputs of every call are as alone."""
    import threading
    jobs, errors = [], []
    for i in range(6):
        gen = torch.Generator().manual_seed(190 + i)
        lens = [70 * i + 1, 1900 - 300 * i, 17]
        kind = ("bf16", "fp16", "e4m3")[i % 3]
        table, pages = R.table_for(lens, 16, gen)
        pool = R.Pool(kind, pages, 16, 2, 64, "rows", gen)
        q = torch.randn(3, 8, 64, generator=gen).to(torch.float16 if kind == "fp16" else torch.bfloat16)
        jobs.append((pool.on_gpu(), q.cuda(), table.cuda(), _i32(lens), max(lens), R.attention(q, pool, table, lens, 16)))
    torch.cuda.synchronize()

    def work(cache, q, table, lens, most, ref):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(8):
                    w, lse = torch.zeros(3, 2, most, device="cuda"), torch.zeros(3, 8, device="cuda")
                    out = L.tc_paged_attention(q, cache, table, lens, weights=w, lse=lse, max_len=most)
                    s.synchronize()
                    for got, want, tol in ((w, ref[2], ref[5] + 2 * R.STEP32 * ref[2]), (lse, ref[1], ref[4]),
                                           (out, ref[0], ref[3] + _half_step(q.dtype, ref[0], ref[3]))):
                        assert bool(((got.cpu().double() - want).abs() <= tol).all())
        except BaseException as e:  # reported below
            errors.append(repr(e))

    say(f"[gpu] {len(jobs)} threads with weights")
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:2]


@pytest.mark.parametrize("kind, values", [("bf16", (2.0 ** -133, 2.0 ** -127, 1e-37, 1e-30, 1.5e38)),
                                          ("fp16", (2.0 ** -24, 3 * 2.0 ** -24, 2.0 ** -14, 65504.0))])
def test_attention_over_values_at_the_ends_of_their_range(kind, values):
    """Equal values under equal weights: out is the value, of subnormal numbers too, as long as the sum of the values times
    exp(x_i - max x), here their number, stays in fp32's range."""
    dt = R.DT[kind]
    for value in values:
        for rows in (1, 2, 40, 2000):
            if value * rows > 3.4e38:
                continue
            say(f"[gpu] {rows} rows of {value} in {kind}")
            v = torch.full((rows, 32), value).to(dt)
            out = L.tc_paged_attention(*_one_sequence(torch.zeros(rows, 32, dtype=dt), v, torch.ones(2, 32, dtype=dt)))
            assert bool((out.cpu() == v[0]).all()), out[0, 0, 0]
