"""Paged caches for the tests and their operators in 64 bits on the host, written from the definitions."""

import math

import torch

TINY = torch.finfo(torch.float32).tiny
STEP32 = 2.0 ** -24  # half a step of fp32 at 1
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


def bits(x):
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


def quantise(x):
    """e4m3 codes and fp32 scales of the rows of x (last axis), the definition evaluated in fp32."""
    x = x.float()
    scale = x.abs().amax(-1) / 448.0
    scale = torch.where(scale < TINY, torch.ones_like(scale), scale)
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


class Pool:
    """A pool on the host: tensors of logical shape (pages, page, heads, dim), laid out as `major` says."""

    def __init__(self, kind, pages, page, heads, dim, major="rows", gen=None, fill=None):
        shape = {"rows": (pages, page, heads, dim), "heads": (pages, heads, page, dim),
                 "pairs": (pages, 2, page, heads, dim)}[major]
        self.kind, self.major = kind, major

        def make(sh):
            if fill is not None:
                x = torch.full(sh, fill, dtype=torch.float32)
            else:
                x = torch.randn(sh, generator=gen)
            if kind != "e4m3":
                return x.to(DT[kind]), None
            if fill is not None:
                return x.to(DT[kind]), torch.full(sh[:-1], fill, dtype=torch.float32)
            return quantise(x)

        if major == "pairs":  # keys and values of a page side by side in one allocation
            x, s = make(shape)
            self.base = [x] + ([s] if s is not None else [])
            self.k, self.v = x[:, 0], x[:, 1]
            self.ks, self.vs = (None, None) if s is None else (s[:, 0], s[:, 1])
        else:
            k, ks = make(shape)
            v, vs = make(shape)
            if major == "heads":
                k, v = k.transpose(1, 2), v.transpose(1, 2)
                ks, vs = (None, None) if ks is None else (ks.transpose(1, 2), vs.transpose(1, 2))
            self.k, self.v, self.ks, self.vs = k, v, ks, vs

    def tensors(self):
        return [x for x in (self.k, self.v, self.ks, self.vs) if x is not None]

    def on_gpu(self):
        """The same pool on the GPU, with the same strides, and the cache over it."""
        import layout_permuting_copy_amd as L
        if self.major == "pairs":
            base = [b.cuda() for b in self.base]
            k, v = base[0][:, 0], base[0][:, 1]
            ks, vs = (base[1][:, 0], base[1][:, 1]) if len(base) > 1 else (None, None)
        else:
            k, v, ks, vs = (None if x is None else
                            (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.major == "heads"
                             else x.contiguous().cuda())
                            for x in (self.k, self.v, self.ks, self.vs))
        return L.PagedCache(k, v, ks, vs)

    def rows(self, which, table_row, n, page):
        """Rows 0 .. n - 1 of a sequence in fp64, (n, heads, dim), and whether each lies on a page."""
        x, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        i = torch.arange(n)
        pg = table_row[i // page].long()
        ok = (pg >= 0) & (pg < x.shape[0])
        pg = torch.where(ok, pg, torch.zeros_like(pg))
        y = bits(x)[pg, i % page].view(x.dtype).float().double()
        if s is not None:
            y = y * s[pg, i % page].double().unsqueeze(-1)
        return y, ok


def cache_tensors(cache):
    return [x for x in (cache.k, cache.v, cache.k_scale, cache.v_scale) if x is not None]


def table_for(lens, page, gen, cols=None, spare=0, junk=-1):
    """A block table over randomly ordered pages, `junk` past each sequence's end, and the pool's pages."""
    need = [(n + page - 1) // page for n in lens]
    pages = max(1, sum(need)) + spare
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need, default=1)) if cols is None else cols), junk, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    return table, pages


def attention(q, pool, table, lens, page, scale=None):
    """out, lse, p of every cache row (batch, heads, longest), and the bounds that the kernel's fp32 steps stay
    within: tolerances for out (before its rounding), lse and p.

    With e = 2^-24 a product or sum in fp32 is off by e relative to its terms.  A logit sums D products (exact
    in fp32, or off by e) and takes two factors: off by dx = (D + 8) e scale sum |q k| at most, e for the base-2
    factor and the exponential's own error (2 units, 4 e) beside it.  A weight is off by the relative amount
    exp(dx) - 1, from its own logit and from the row's maximum and sum: 2 dx + 16 e.  Sums over rows run to
    a depth of n / 16 + 96 additions (waves, tiles, splits), each off by e of the sum of magnitudes.  The weights
    enter the second product as two 16-bit values: bf16 leaves 2^-17 of the weight, fp16 2^-22 of it or 2^-40 of
    the row's maximum (whose weight before division is 2^15)."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    batch, heads_q, dim = q.shape
    heads = pool.k.shape[2]
    group = heads_q // heads
    longest = max(max(lens), 1)
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    weight = torch.zeros(batch, heads, longest, dtype=torch.float64)
    t_out, t_lse, t_w = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(weight)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, ok = pool.rows("k", table[b], n, page)
        v, _ = pool.rows("v", table[b], n, page)
        if not ok.any():
            continue
        at = torch.nonzero(ok)[:, 0]
        k, v = k[at], v[at]
        depth = (n / 16 + 96) * STEP32
        for hq in range(heads_q):
            h = hq // group
            x = k[:, h] @ q[b, hq].double() * scale
            if not (x > -math.inf).any() and not x.isnan().any():
                continue
            dx = (dim + 8) * STEP32 * (k[:, h].abs() @ q[b, hq].double().abs()).max() * abs(scale)
            total = torch.logsumexp(x, 0)
            p = torch.exp(x - total)
            rel = 2 * dx + 16 * STEP32 + depth
            out[b, hq] = p @ v[:, h]
            lse[b, hq] = total
            weight[b, h, at] += p
            mag = p @ v[:, h].abs()
            t_out[b, hq] = mag * (rel + 2.0 ** -17)
            if q.dtype == torch.float16 and pool.kind != "e4m3":
                t_out[b, hq] += 2.0 ** -40 * torch.exp(x.max() - total) * v[:, h].abs().sum(0)
            t_lse[b, hq] = dx + 16 * STEP32 + depth + 4 * STEP32 * (abs(total) + abs(x).max())
            t_w[b, h, at] += p * rel
    return out, lse, weight, t_out, t_lse, t_w


def keep_rows(w, n, budget, recent):
    """Rows of one head that stay, ascending: the recent ones, then by weight (NaN first), then the lowest."""
    if n <= budget:
        return list(range(n))
    old = n - recent
    rank = sorted(range(old), key=lambda i: ((0, 0.0) if math.isnan(w[i]) else (1, -w[i]), i))
    return sorted(rank[:budget - recent]) + list(range(old, n))
