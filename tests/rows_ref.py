"""Attention of several query rows a sequence in 64 bits on the host, with the bounds that the kernels stay within."""

import math

import torch

STEP32 = 2.0 ** -24  # half a step of fp32 at 1


def sequence(q, k, v, seen, scale=None, part=None):
    """q (n, q_heads, dim) over k, v (m, heads, dim) in fp64, `seen` (n, m) bool: out, lse and tolerances for out (before its
    rounding) and lse.

    With e = 2^-24: a logit sums dim products and takes a factor, dx = (dim + 8) e scale sum |q k| at most; a weight is off by
    the relative amount 2 dx + 16 e, from its own logit, the exponential and the reference.  A lane adds up to m / 2 weights one
    after another, the matrix unit a tile's products to its sum: m / 2 + 96 steps of e each, relative to the sum of
    magnitudes, for parts of the keys and their join too.  A weight enters the second product as a 16-bit value, off by
    `part` of it at most (half a step of its type; its square for two values), and, in fp16, by 2^-32 of the row's
    greatest: that is held as 2^7 or more, and half a step of a subnormal is 2^-25."""
    n, q_heads, dim = q.shape
    m, heads, _ = k.shape
    scale = dim ** -0.5 if scale is None else scale
    out, lse = torch.zeros(q.shape, dtype=torch.float64), torch.full((n, q_heads), -math.inf, dtype=torch.float64)
    t_out, t_lse = torch.zeros_like(out), torch.zeros_like(lse)
    if n == 0 or m == 0:
        return out, lse, t_out, t_lse
    subnormal = 2.0 ** -32 if q.dtype == torch.float16 and k.dtype == torch.float16 else 0.0
    if part is None:
        part = half_step(k.dtype)
    q, k, v = q.double(), k.double(), v.double()
    depth = (m / 2 + 96) * STEP32
    for hq in range(q_heads):
        h = hq // (q_heads // heads)
        # what is not seen does not count, whatever it is
        use = seen.any(0)
        kh, vh = k[use, h], v[use, h]
        see = seen[:, use]
        x = (q[:, hq] @ kh.T * scale).masked_fill(~see, -math.inf)
        size = (q[:, hq].abs() @ kh.abs().T * abs(scale)).masked_fill(~see, 0.0)
        size = torch.nan_to_num(size, nan=0.0, posinf=0.0)
        dx = (dim + 8) * STEP32 * size.amax(1) if size.shape[1] else torch.zeros(n, dtype=torch.float64)
        total = torch.logsumexp(x, 1) if x.shape[1] else torch.full((n,), -math.inf, dtype=torch.float64)
        some = total > -math.inf
        some |= total.isnan()
        p = torch.exp(x - total.masked_fill(~some, 0.0)[:, None]).masked_fill(~see, 0.0)
        for i in range(n):
            if not some[i]:
                continue
            out[i, hq] = p[i, see[i]] @ vh[see[i]]
            mag = p[i, see[i]] @ vh[see[i]].abs()
            t_out[i, hq] = mag * (2 * dx[i] + 16 * STEP32 + 2 * depth + part)
            t_out[i, hq] += subnormal * p[i].max() * vh[see[i]].abs().sum(0)
        lse[:, hq] = total
        t_lse[:, hq] = dx + 16 * STEP32 + depth + 4 * STEP32 * (torch.nan_to_num(total, neginf=0.0).abs() +
                                                               torch.nan_to_num(x, neginf=0.0, posinf=0.0).abs().amax(1) if x.shape[1] else 0.0)
    return out, lse, t_out, t_lse


def half_step(dtype):
    return torch.finfo(torch.float16 if dtype == torch.float16 else torch.bfloat16).eps / 2


def before(n, m):
    """Which of m rows the last n of them see, causally."""
    return torch.arange(m)[None, :] <= (torch.arange(n) + m - n)[:, None]


def by_masks(masks, n, m):
    """Which of m rows the last n see: those before these n, and of these the ones that a token's word names."""
    seen = torch.ones(n, m, dtype=torch.bool)
    for i in range(n):
        for j in range(n):
            if m - n + j >= 0:
                seen[i, m - n + j] = j < 64 and bool(int(masks[i]) >> j & 1)
    return seen


def close(got, want, tol, what, out_dtype=None):
    got = got.cpu().double()
    if out_dtype is not None:  # out's own rounding
        f = torch.finfo(out_dtype)
        tol = tol + f.eps / 2 * (want.abs() + tol).clamp_min(f.smallest_normal)
    fine = (got.isnan() & want.isnan()) | (got == want) | ((got - want).abs() <= tol)
    if not bool(fine.all()):
        at = tuple(torch.nonzero(~fine)[0].tolist())
        raise AssertionError(f"{what}: {int((~fine).sum())} of {fine.numel()} off; at {at} got {got[at]} want {want[at]} "
                             f"tolerance {tol[at]}")


def starts_of(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def resize(table, lens, change, stack, count, page, tokens):
    """Lists in, lists out: (table, lens, stack, count, missing, starts, slots, positions)."""
    most = 2 ** 31 - 1
    table, stack = [list(r) for r in table], list(stack)
    cols, cap = len(table[0]) if table else 0, len(stack)
    count = max(0, min(count, cap))
    pages = lambda n: min(-(-n // page), cols)
    lens = [max(0, n) for n in lens]
    new = [max(0, min(n + c, most)) for n, c in zip(lens, change)]
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in range(pages(m), pages(n)):
            if table[b][i] >= 0 and count < cap:
                stack[count] = table[b][i]
                count += 1
    missing = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in range(pages(n), pages(m)):
            if count:
                count -= 1
                table[b][i] = stack[count]
            else:
                table[b][i] = -1
                missing += 1
    starts, slots, positions = [0], [], []
    for b, (n, m) in enumerate(zip(lens, new)):
        grown = max(0, m - n)
        starts.append(min(starts[-1] + grown, most))
        for row in range(n, n + min(grown, max(0, tokens - len(slots)))):
            at = table[b][row // page] if row // page < cols else -1
            slots.append(at * page + row % page if at >= 0 else -1)
            positions.append(row)
    slots += [-1] * (tokens - len(slots))
    positions += [-1] * (tokens - len(positions))
    return table, new, stack, count, missing, starts, slots[:tokens], positions[:tokens]
