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
