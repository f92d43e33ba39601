"""Workloads of the paged key-value cache operators: append, attention of one new token, eviction.

``listed()`` names the cases, ``draw()`` makes more of the same ranges, ``prepare()`` makes what a
serving loop holds before the call, ``run()`` is one pass through an operator: its plain form in
elementary torch operations (``own = False``) or the library's entry point (``own = True``).
``exact()`` evaluates the definition in 64 bits, ``work()`` counts the bytes and operations a pass
cannot do without.

A cache is a pool of pages, logical shape (pages, page_size, heads, head_dim) for keys and for
values; a block table names each sequence's pages in order.  8-bit caches hold e4m3 codes and one
fp32 scale a row and head: scale = amax / 448 (1 where that is below the smallest normal fp32),
code = value / scale rounded to nearest even.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
TINY = torch.finfo(torch.float32).tiny
GOLDEN = 0.6180339887498949


# ---- the cases -------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's keys and values of 32 sequences entering the cache (a launch's latency)
        dict(name="append_step", op="append", dtype="bf16", cache="bf16", batch=32, chunk=1, spread="step",
             kv_heads=8, head_dim=128, page=16, major="rows", fused=True),
        # prompts of unequal lengths, their keys and values sliced out of a fused projection's rows
        dict(name="append_prompts", op="append", dtype="bf16", cache="bf16", batch=9, chunk=4095, spread="ragged",
             kv_heads=8, head_dim=128, page=16, major="rows", fused=True),
        # chunks of prompts quantised to 8 bits on their way into pages that keep a head's rows together
        dict(name="append_chunks_8bit", op="append", dtype="fp16", cache="e4m3", batch=16, chunk=1021,
             spread="ragged", kv_heads=8, head_dim=64, page=64, major="heads", fused=False),
        # one chat at its beginning: a short cache, where the call's latency is everything
        dict(name="attend_short", op="attend", dtype="bf16", cache="bf16", batch=1, length=131, spread="full",
             q_heads=32, kv_heads=8, head_dim=128, page=16, major="rows", weights=False),
        # a serving batch at mixed lengths, some sequences just begun and one slot empty
        dict(name="attend_batch", op="attend", dtype="bf16", cache="bf16", batch=64, length=4096, spread="ragged",
             q_heads=32, kv_heads=8, head_dim=128, page=16, major="rows", weights=False),
        # one long document: few rows, so the cache's length itself has to fill the chip
        dict(name="attend_long", op="attend", dtype="bf16", cache="bf16", batch=1, length=131072, spread="full",
             q_heads=64, kv_heads=8, head_dim=128, page=64, major="heads", weights=False),
        # as many key heads as query heads, small heads, pages that are no power of two
        dict(name="attend_odd_pages", op="attend", dtype="fp16", cache="fp16", batch=24, length=2047, spread="ragged",
             q_heads=16, kv_heads=16, head_dim=64, page=24, major="rows", weights=False),
        # the largest: a batch of long sequences in an 8-bit cache
        dict(name="attend_8bit", op="attend", dtype="bf16", cache="e4m3", batch=32, length=16384, spread="full",
             q_heads=64, kv_heads=8, head_dim=128, page=32, major="heads", weights=False),
        # decoding under a cache budget: the step also adds its attention weights up for the eviction
        dict(name="attend_weights", op="attend", dtype="bf16", cache="bf16", batch=8, length=8192, spread="ragged",
             q_heads=32, kv_heads=8, head_dim=128, page=16, major="rows", weights=True),
        # one shared key head of 256 elements under 16 query heads
        dict(name="attend_one_kv_head", op="attend", dtype="fp16", cache="fp16", batch=16, length=5000,
             spread="ragged", q_heads=16, kv_heads=1, head_dim=256, page=16, major="rows", weights=False),
        # one sequence over its budget
        dict(name="evict_one", op="evict", cache="fp16", batch=1, length=2049, spread="full", budget=1024, recent=128,
             kv_heads=8, head_dim=128, page=16, major="rows"),
        # a batch shrunk after its prompts: long rows of weights, most of the cache dropped
        dict(name="evict_batch", op="evict", cache="bf16", batch=16, length=16384, spread="ragged", budget=4096,
             recent=512, kv_heads=8, head_dim=128, page=16, major="rows"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict"])
    dtype = rng.choice(["bf16", "fp16"])
    case = dict(op=op, cache=rng.choice([dtype, dtype, "e4m3"]), kv_heads=rng.choice([1, 2, 3, 4, 5, 8, 16]),
                head_dim=rng.choice([32, 64, 80, 96, 128, 128, 192, 256]), page=rng.choice([1, 8, 16, 16, 24, 32, 64, 100]),
                major=rng.choice(["rows", "heads"]))
    row = case["kv_heads"] * case["head_dim"] * 4
    if op == "append":
        case["dtype"] = dtype
        case["batch"] = _log_int(rng, 1, 64)
        case["spread"] = rng.choice(["step", "ragged"])
        most = max(2, min(4096, 128 * 2**20 // (row * case["batch"])))
        case["chunk"] = 1 if case["spread"] == "step" else _log_int(rng, 2, most)
        case["fused"] = rng.random() < 0.5
    elif op == "attend":
        case["dtype"] = dtype
        case["batch"] = _log_int(rng, 1, 64)
        case["spread"] = rng.choice(["full", "ragged"])
        case["length"] = _log_int(rng, 1, max(1, min(131072, 512 * 2**20 // (row * case["batch"]))))
        case["q_heads"] = case["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 20])
        case["weights"] = rng.random() < 0.3
    else:
        case["batch"] = _log_int(rng, 1, 16)
        case["spread"] = rng.choice(["full", "ragged"])
        case["length"] = _log_int(rng, 2, max(2, min(65536, 256 * 2**20 // (row * case["batch"]))))
        case["budget"] = rng.randint(1, case["length"] + case["length"] // 8)
        case["recent"] = rng.randint(0, min(case["budget"], 512))
    return case


def _lengths(case):
    """Lengths of the cache, or of the chunks that enter it: a rule of the case alone."""
    n, b = case.get("length", case.get("chunk")), case["batch"]
    if case["spread"] != "ragged":
        return [n] * b
    out = [max(1, math.ceil(n * math.modf((i + 1) * GOLDEN)[0])) for i in range(b)]
    for i in range(b):
        if i % 11 == 5:
            out[i] = 0
        elif i % 13 == 7:
            out[i] = 1
    out[b // 2] = n
    return out


def _before(case):
    """Rows that the cache holds before an append."""
    return [(37 * i) % 97 for i in range(case["batch"])]


# ---- inputs ----------------------------------------------------------------------------------

def _quantise(x):
    """e4m3 codes and the fp32 scale of each row (the last axis)."""
    x = x.float()
    scale = x.abs().amax(-1) / 448.0
    scale = torch.where(scale < TINY, torch.ones_like(scale), scale)
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _pool(case, pages, gen, fill):
    """Keys or values of a pool of pages, logical (pages, page, heads, head_dim), and the scales."""
    heads, dim, page = case["kv_heads"], case["head_dim"], case["page"]
    by_heads = case["major"] == "heads"
    shape = (pages, heads, page, dim) if by_heads else (pages, page, heads, dim)
    dtype, scale = DTYPES[case["cache"]], None
    if not fill:
        x = torch.zeros(shape, dtype=torch.uint8 if case["cache"] == "e4m3" else dtype, device="cuda").view(dtype)
        if case["cache"] == "e4m3":
            scale = torch.zeros(shape[:3], device="cuda")
    else:
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        if case["cache"] == "e4m3":
            x, scale = _quantise(x)
        else:
            x = x.to(dtype)
    if by_heads:
        x = x.transpose(1, 2)
        scale = None if scale is None else scale.transpose(1, 2)
    return x, scale


def _table(lens, page, gen, width=None):
    """A block table whose pages lie anywhere in the pool; entries past a sequence's end are -1."""
    need = [(n + page - 1) // page for n in lens]
    width = max(1, max(need)) if width is None else width
    pages = max(1, sum(need))
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = order[at:at + c]
        at += c
    return table, pages


def _cache(state, name, k, v, ks, vs):
    state[name] = dict(k=k, v=v, ks=ks, vs=vs)
    if own:
        import layout_permuting_copy_amd as L
        state[name]["handle"] = L.PagedCache(k, v, ks, vs)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = _lengths(case)
    batch, page, heads, dim = case["batch"], case["page"], case["kv_heads"], case["head_dim"]
    state = dict(case=case, op=case["op"])
    if case["op"] == "append":
        dtype = DTYPES[case["dtype"]]
        total = [a + b for a, b in zip(_before(case), lens)]
        tokens = sum(lens)
        if case["fused"]:  # the rows of a projection to two query heads a key head, keys and values
            rows = torch.randn(tokens, 4 * heads * dim, generator=gen, device="cuda", dtype=dtype)
            state["k_new"] = rows[:, 2 * heads * dim:3 * heads * dim].unflatten(1, (heads, dim))
            state["v_new"] = rows[:, 3 * heads * dim:].unflatten(1, (heads, dim))
        else:
            state["k_new"] = torch.randn(tokens, heads, dim, generator=gen, device="cuda", dtype=dtype)
            state["v_new"] = torch.randn(tokens, heads, dim, generator=gen, device="cuda", dtype=dtype)
        table, pages = _table(total, page, gen)
        k, ks = _pool(case, pages, gen, False)
        v, vs = _pool(case, pages, gen, False)
        _cache(state, "cache", k, v, ks, vs)
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        state.update(table=table, lens_host=total, chunk_host=lens,
                     lens=torch.tensor(total, dtype=torch.int32, device="cuda"),
                     starts=None if case["spread"] == "step" else torch.tensor(starts, dtype=torch.int32, device="cuda"))
        return state
    table, pages = _table(lens, page, gen)
    k, ks = _pool(case, pages, gen, True)
    v, vs = _pool(case, pages, gen, True)
    _cache(state, "cache", k, v, ks, vs)
    state.update(table=table, lens_host=lens, max_len=max(lens),
                 lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["op"] == "attend":
        dtype = DTYPES[case["dtype"]]
        # logits of standard deviation 2.5: some rows are sharp, some flat
        state["q"] = (2.5 * torch.randn(batch, case["q_heads"], dim, generator=gen, device="cuda")).to(dtype)
        state["lse"] = torch.empty(batch, case["q_heads"], device="cuda")
        if case["weights"]:
            state["weights"] = 4.0 * torch.rand(batch, heads, state["max_len"], generator=gen, device="cuda")
            state["weights_out"] = state["weights"].clone()
    else:
        # sums of attention weights: heavy tails, rows never attended to, equal values
        w = torch.exp(2.0 * torch.randn(batch, heads, state["max_len"], generator=gen, device="cuda"))
        u = torch.rand(w.shape, generator=gen, device="cuda")
        w = torch.where(u < 0.1, torch.zeros_like(w), torch.where(u < 0.4, torch.floor(w * 64.0) / 64.0, w))
        budget = case["budget"]
        kept = [min(n, budget) for n in lens]
        dst_table, dst_pages = _table(kept, page, gen)
        dk, dks = _pool(case, dst_pages, gen, False)
        dv, dvs = _pool(case, dst_pages, gen, False)
        _cache(state, "into", dk, dv, dks, dvs)
        most = max(1, max(kept))
        state.update(weights=w, into_table=dst_table, kept=torch.zeros(batch, heads, most, dtype=torch.int32, device="cuda"),
                     weights_out=torch.zeros(batch, heads, most, device="cuda"),
                     lens_out=torch.zeros(batch, dtype=torch.int32, device="cuda"))
    return state


# ---- one pass --------------------------------------------------------------------------------

def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _where(table_row, first, n, page):
    i = torch.arange(first, first + n, device="cuda")
    return table_row[i // page].long(), i % page


def _plain_append(s):
    c, page = s["cache"], s["case"]["page"]
    pages, rows = [], []
    for b, n in enumerate(s["chunk_host"]):
        p, r = _where(s["table"][b], s["lens_host"][b] - n, n, page)
        pages.append(p)
        rows.append(r)
    pages, rows = torch.cat(pages), torch.cat(rows)
    for pool, scales, new in ((c["k"], c["ks"], s["k_new"]), (c["v"], c["vs"], s["v_new"])):
        if scales is None:
            pool[pages, rows] = new
        else:
            code, scale = _quantise(new)
            _bits(pool)[pages, rows] = _bits(code)
            scales[pages, rows] = scale


def _plain_rows(pool, scales, pages, rows):
    x = _bits(pool)[pages, rows].view(pool.dtype).float()
    return x if scales is None else x * scales[pages, rows].unsqueeze(-1)


def _plain_attend(s):
    c, case = s["cache"], s["case"]
    heads, dim, group = case["kv_heads"], case["head_dim"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros_like(s["q"])
    s["lse"].fill_(-math.inf)
    for b, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        at = _where(s["table"][b], 0, n, case["page"])
        k = _plain_rows(c["k"], c["ks"], *at).permute(1, 2, 0).contiguous()
        v = _plain_rows(c["v"], c["vs"], *at).transpose(0, 1).contiguous()
        x = torch.matmul(s["q"][b].float().view(heads, group, dim), k) / math.sqrt(dim)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        p = p / total
        out[b] = torch.matmul(p, v).view(-1, dim).to(out.dtype)
        s["lse"][b] = (top + torch.log(total)).view(-1)
        if case["weights"]:
            s["weights_out"][b, :, :n] = s["weights"][b, :, :n] + p.sum(1)
    return out


def _plain_evict(s):
    c, d, case = s["cache"], s["into"], s["case"]
    page, budget = case["page"], case["budget"]
    head = torch.arange(case["kv_heads"], device="cuda").unsqueeze(1)
    s["kept"].fill_(-1)
    for b, n in enumerate(s["lens_host"]):
        new = min(n, budget)
        s["lens_out"][b] = new
        if new == 0:
            continue
        if n <= budget:
            keep = torch.arange(n, device="cuda").repeat(case["kv_heads"], 1)
        else:
            old = n - case["recent"]
            order = torch.sort(s["weights"][b, :, :old], dim=-1, descending=True, stable=True).indices
            late = torch.arange(old, n, device="cuda").repeat(case["kv_heads"], 1)
            keep = torch.cat([order[:, :budget - case["recent"]], late], 1).sort(-1).values
        src = s["table"][b][keep // page].long()
        at = torch.arange(new, device="cuda")
        dst, row = s["into_table"][b][at // page].long().unsqueeze(0), (at % page).unsqueeze(0)
        for x, y in (("k", "ks"), ("v", "vs")):
            _bits(d[x])[dst, row, head] = _bits(c[x])[src, keep % page, head]
            if c[y] is not None:
                d[y][dst, row, head] = c[y][src, keep % page, head]
        s["kept"][b, :, :new] = keep.to(torch.int32)
        s["weights_out"][b, :, :new] = torch.gather(s["weights"][b], 1, keep)


def _pool_outputs(c):
    return [x for x in (c["k"], c["v"], c["ks"], c["vs"]) if x is not None]


def run(state):
    s = state
    if own:
        import layout_permuting_copy_amd as L
    if s["op"] == "append":
        if own:
            L.tc_paged_append(s["cache"]["handle"], s["k_new"], s["v_new"], s["table"], s["lens"], token_starts=s["starts"])
        else:
            _plain_append(s)
        return _pool_outputs(s["cache"])
    if s["op"] == "attend":
        if own:
            out = L.tc_paged_attention(s["q"], s["cache"]["handle"], s["table"], s["lens"], max_len=s["max_len"],
                                       lse=s["lse"], weights=s.get("weights"), weights_out=s.get("weights_out"))
        else:
            out = _plain_attend(s)
        return [out, s["lse"]] + ([s["weights_out"]] if "weights" in s else [])
    if own:
        L.tc_paged_evict(s["cache"]["handle"], s["table"], s["lens"], s["weights"], s["into"]["handle"], s["into_table"],
                         s["case"]["budget"], s["case"]["recent"], max_len=s["max_len"], lens_out=s["lens_out"],
                         weights_out=s["weights_out"], kept=s["kept"])
    else:
        _plain_evict(s)
    return [s["lens_out"], s["kept"], s["weights_out"]] + _pool_outputs(s["into"])


# ---- the definitions in 64 bits --------------------------------------------------------------

def _slots(table_row, n, page):
    """Pool rows (page * page_size + offset) of a sequence's first n cache rows, on the host."""
    i = np.arange(n)
    return table_row[i // page].astype(np.int64) * page + i % page


def _flat(x):
    """A pool as 64-bit rows (pages * page_size, heads, ...); 8-bit codes as the values they stand for."""
    return (x.float() if x.dtype == torch.float8_e4m3fn else x).double().reshape(-1, *x.shape[2:])


def _exact_append(case, s):
    table = s["table"].cpu().numpy()
    slots = np.concatenate([_slots(table[b], t, case["page"])[t - n:]
                            for b, (t, n) in enumerate(zip(s["lens_host"], s["chunk_host"]))])
    slots = torch.from_numpy(slots).cuda()
    pools, scales = [], []
    for name, new in (("k", s["k_new"]), ("v", s["v_new"])):
        pool, x = s["cache"][name], new.double()
        rows = torch.zeros(pool.shape[0] * pool.shape[1], *pool.shape[2:], dtype=torch.float64, device="cuda")
        if case["cache"] == "e4m3":
            scale = x.abs().max(-1).values / 448.0
            scale[scale < TINY] = 1.0
            x = x / scale[..., None]
            held = torch.zeros(rows.shape[:2], dtype=torch.float64, device="cuda")
            held[slots] = scale
            scales.append(held.reshape(pool.shape[:3]))
        rows[slots] = x
        pools.append(rows.reshape(pool.shape))
    return pools + scales


def _exact_attend(case, s):
    table, c = s["table"].cpu().numpy(), s["cache"]
    group, dim = case["q_heads"] // case["kv_heads"], case["head_dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    weights = s["weights_out"].double() if case["weights"] else None
    for b, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        slots = torch.from_numpy(_slots(table[b], n, case["page"])).cuda()
        page, row = slots // case["page"], slots % case["page"]
        for h in range(case["kv_heads"]):
            k, v = (_bits(c[x])[page, row, h].view(c[x].dtype).float().double() for x in ("k", "v"))
            if c["ks"] is not None:
                k = k * c["ks"][page, row, h].double()[:, None]
                v = v * c["vs"][page, row, h].double()[:, None]
            q = s["q"][b, h * group:(h + 1) * group].double()
            x = (k @ q.T).T * dim ** -0.5
            total = torch.logsumexp(x, 1)
            p = torch.exp(x - total[:, None])
            out[b, h * group:(h + 1) * group] = p @ v
            lse[b, h * group:(h + 1) * group] = total
            if weights is not None:
                weights[b, h, :n] = s["weights"][b, h, :n].double() + p.sum(0)
    return [out, lse] + ([weights] if weights is not None else [])


def _exact_evict(case, s):
    table, into = s["table"].cpu().numpy(), s["into_table"].cpu().numpy()
    w = s["weights"].cpu().numpy()
    kept = np.full(tuple(s["kept"].shape), -1, dtype=np.int32)
    weights = np.zeros(kept.shape)
    lens = np.zeros(case["batch"], dtype=np.int32)
    names = [x for x in ("k", "v", "ks", "vs") if s["cache"][x] is not None]
    src = [_flat(s["cache"][x]) for x in names]
    dst = [_flat(s["into"][x]) for x in names]
    for b, n in enumerate(s["lens_host"]):
        lens[b] = new = min(n, case["budget"])
        if new == 0:
            continue
        from_slots, to_slots = _slots(table[b], n, case["page"]), _slots(into[b], new, case["page"])
        for h in range(case["kv_heads"]):
            # rows by descending rank: the recent ones, then the heaviest, then the earliest
            i = np.arange(n)
            rank = np.lexsort((i, -w[b, h, :n].astype(np.float64), i < n - case["recent"]))
            keep = np.sort(rank[:new])
            kept[b, h, :new], weights[b, h, :new] = keep, w[b, h, keep]
            a, z = torch.from_numpy(from_slots[keep]).cuda(), torch.from_numpy(to_slots).cuda()
            for x, y in zip(src, dst):
                y[z, h] = x[a, h]
    pools = [y.reshape(s["into"][x].shape) for x, y in zip(names, dst)]
    return [torch.from_numpy(lens).cuda(), torch.from_numpy(kept).cuda(), torch.from_numpy(weights).cuda()] + pools


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](case, s)


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    lens, page, heads, dim = _lengths(case), case["page"], case["kv_heads"], case["head_dim"]
    quantised = case["cache"] == "e4m3"
    row = 2 * heads * ((dim + 4) if quantised else 2 * dim)  # a token's keys and values, scales among them
    if case["op"] == "append":
        tables = sum(-(-(a + n) // page) - a // page for a, n in zip(_before(case), lens))
        flops = sum(lens) * 2 * heads * dim * 3 if quantised else 0  # magnitude, maximum, division
        return {"bytes": sum(lens) * (4 * heads * dim + row) + 4 * (tables + 2 * len(lens)), "flops": flops}
    tables = 4 * (sum(-(-n // page) for n in lens) + len(lens))
    if case["op"] == "attend":
        small = len(lens) * case["q_heads"] * (2 * 2 * dim + 4) + tables
        weights = 8 * sum(lens) * heads if case["weights"] else 0
        return {"bytes": sum(lens) * row + small + weights, "flops": 4 * sum(lens) * case["q_heads"] * dim}
    new = [min(n, case["budget"]) for n in lens]
    scored = sum((n - case["recent"]) if n > case["budget"] else 0 for n in lens)
    small = tables + 4 * (sum(-(-n // page) for n in new) + len(lens))
    return {"bytes": 2 * sum(new) * row + 4 * heads * (scored + 3 * sum(new)) + small, "flops": scored * heads}
