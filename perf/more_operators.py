"""Workloads of a serving step's operators beside the paged cache: growing and shrinking the block tables, attention over
whole prompts, attention of several new tokens a sequence (drafted trees, chunks of prompts) over the cache.

``listed()`` names the cases, ``draw()`` makes more of the same ranges, ``prepare()`` makes what a
serving loop holds before the call, ``run()`` is one pass through an operator: its plain form in
elementary torch operations (``own = False``) or the library's entry point (``own = True``).
``exact()`` evaluates the definition in 64 bits, ``work()`` counts the bytes and operations a pass
cannot do without.

resize   sequence b goes from n to max(0, n + change[b]) rows: the pages it no longer needs go onto a stack of free
         pages, then the pages that others need come off it, sequence by sequence; each new row's place in the pool
         (its slot, page * page_size + row of the page) and position in its sequence are listed
prompt   softmax(scale q k^T) v over packed sequences, causal or not, query heads in groups over key heads; the
         queries are the last tokens of the keys' sequence where there are more keys
tree     the same of each sequence's last tokens over its cache: a drafted token sees the rows before the draft and
         the drafted tokens that bits of its mask name; without masks those before it (a chunk of a prompt)
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
        # one decode step's bookkeeping of 48 sequences: a new row each, some finished (a launch's latency)
        dict(name="resize_step", op="resize", batch=48, length=2048, chunk=1, page=16, short=False),
        # a step that takes in prompts, rejects drafts and lets sequences go
        dict(name="resize_prompts", op="resize", batch=192, length=8192, chunk=4095, page=16, short=False),
        # one chat's first prompt: latency
        dict(name="prompt_short", op="prompt", dtype="bf16", batch=1, length=131, prefix=0, spread="full", causal=True,
             q_heads=32, kv_heads=8, head_dim=128, fused=True, pad=0),
        # prompts of unequal lengths packed into one call, sliced out of a fused projection's rows, and padding behind
        dict(name="prompt_packed", op="prompt", dtype="bf16", batch=13, length=4095, prefix=0, spread="ragged",
             causal=True, q_heads=32, kv_heads=8, head_dim=128, fused=True, pad=37),
        # the largest: one long document
        dict(name="prompt_long", op="prompt", dtype="bf16", batch=1, length=16384, prefix=0, spread="full", causal=True,
             q_heads=32, kv_heads=8, head_dim=128, fused=False, pad=0),
        # later parts of prompts, whose beginnings were computed before, one shared key head of 256
        dict(name="prompt_parts", op="prompt", dtype="fp16", batch=5, length=1000, prefix=3001, spread="ragged",
             causal=True, q_heads=16, kv_heads=1, head_dim=256, fused=False, pad=0),
        # an encoder: every token sees every other, as many key heads as query heads, small odd heads
        dict(name="prompt_encoder", op="prompt", dtype="fp16", batch=24, length=1021, prefix=0, spread="ragged",
             causal=False, q_heads=12, kv_heads=12, head_dim=80, fused=True, pad=0),
        # one chat's drafted tree of 8 tokens: latency
        dict(name="tree_short", op="tree", dtype="bf16", cache="bf16", batch=1, length=523, tokens=8, spread="full",
             q_heads=32, kv_heads=8, head_dim=128, page=16, major="rows", chain=False),
        # a serving batch, trees of unequal sizes over caches of unequal lengths
        dict(name="tree_batch", op="tree", dtype="bf16", cache="bf16", batch=32, length=4096, tokens=26, spread="ragged",
             q_heads=32, kv_heads=8, head_dim=128, page=16, major="rows", chain=False),
        # the largest trees over few long documents: the caches' lengths have to fill the chip
        dict(name="tree_long", op="tree", dtype="bf16", cache="bf16", batch=2, length=65536, tokens=64, spread="full",
             q_heads=64, kv_heads=8, head_dim=128, page=64, major="heads", chain=False),
        # trees over an 8-bit cache
        dict(name="tree_8bit", op="tree", dtype="bf16", cache="e4m3", batch=16, length=8192, tokens=12, spread="full",
             q_heads=64, kv_heads=8, head_dim=128, page=32, major="heads", chain=False),
        # chunks of prompts over what the cache holds of them, pages that are no power of two
        dict(name="tree_chunks", op="tree", dtype="fp16", cache="fp16", batch=4, length=8000, tokens=509, spread="ragged",
             q_heads=16, kv_heads=16, head_dim=64, page=24, major="rows", chain=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["resize", "prompt", "prompt", "tree", "tree"])
    if op == "resize":
        case = dict(op=op, batch=_log_int(rng, 1, 512), length=_log_int(rng, 1, 8192), page=rng.choice([1, 8, 16, 16, 24, 32, 64, 100]))
        case["chunk"] = rng.choice([1, _log_int(rng, 2, 4096)])
        while _grown(case) > _grown(listed()[1]):
            case["chunk"] //= 2
        case["short"] = rng.random() < 0.2
        return case
    most = work(listed()[4])["flops"]
    case = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), batch=_log_int(rng, 1, 32), spread=rng.choice(["full", "ragged"]),
                kv_heads=rng.choice([1, 2, 3, 4, 5, 8, 16]), head_dim=rng.choice([32, 64, 80, 96, 128, 128, 192, 256]))
    group = rng.choice([1, 2, 3, 4, 6, 8, 12])
    case["q_heads"] = case["kv_heads"] * group
    if op == "prompt":
        case.update(length=_log_int(rng, 1, 16384), prefix=rng.choice([0, 0, _log_int(rng, 1, 4096)]),
                    causal=rng.random() < 0.75, fused=rng.random() < 0.5, pad=rng.choice([0, 0, rng.randint(1, 200)]))
    else:
        case.update(cache=rng.choice([case["dtype"], case["dtype"], "e4m3"]), length=_log_int(rng, 1, 65536),
                    chain=rng.random() < 0.3, page=rng.choice([1, 8, 16, 16, 24, 32, 64, 100]),
                    major=rng.choice(["rows", "heads"]))
        case["tokens"] = _log_int(rng, 1, 1024) if case["chain"] else rng.randint(1, 64)
        case["length"] = max(case["length"], case["tokens"])
    rows = max(1, 2**29 // (case["kv_heads"] * case["head_dim"] * 4))  # 512 MB of keys and values
    while work(case)["flops"] > most / 2 or sum(_keys(case)) > rows or _plain_cost(case) > 2**36:
        case["length"] = case["length"] * 3 // 4
        if op == "tree":
            case["tokens"] = max(1, min(case["tokens"], case["length"]))
            case["length"] = max(case["length"], case["tokens"])
        else:
            case["length"] = max(1, case["length"])
            case["prefix"] = case["prefix"] * 3 // 4
    return case


def _plain_cost(case):
    """Elements of all scores: what the plain form writes and reads several times."""
    return sum(n * m for n, m in zip(_queries(case), _keys(case))) * case["q_heads"]


def _spread(n, batch, ragged):
    """Lengths up to n: a rule of the case alone."""
    if not ragged:
        return [n] * batch
    out = [max(1, math.ceil(n * math.modf((i + 1) * GOLDEN)[0])) for i in range(batch)]
    for i in range(batch):
        if i % 11 == 5:
            out[i] = 0
        elif i % 13 == 7:
            out[i] = 1
    out[batch // 2] = n
    return out


def _queries(case):
    """Tokens that ask, by sequence."""
    ragged = case["spread"] == "ragged"
    if case["op"] == "prompt":
        return _spread(case["length"], case["batch"], ragged)
    most = _spread(case["tokens"], case["batch"], ragged)[::-1]
    return [min(a, n) for a, n in zip(most, _spread(case["length"], case["batch"], ragged))]


def _keys(case):
    """Rows that are asked, by sequence."""
    if case["op"] == "tree":
        return _spread(case["length"], case["batch"], case["spread"] == "ragged")
    before = [(case["prefix"] * (i + 1)) // case["batch"] for i in range(case["batch"])]
    return [n + a for n, a in zip(_queries(case), before)]


def _changes(case):
    """Rows that each sequence has and by how many it grows or shrinks."""
    batch, chunk = case["batch"], case["chunk"]
    lens, change = _spread(case["length"], batch, True), []
    for i in range(batch):
        if i % 16 == 3:
            change.append(-lens[i])  # finished
        elif chunk == 1:
            change.append(1)
        elif i % 4 == 0:
            lens[i] = 0  # a new prompt
            change.append(1 + math.ceil((chunk - 1) * math.modf((i + 1) * GOLDEN)[0]))
        elif i % 4 == 1:
            change.append(-min(lens[i], 1 + i % 7))  # drafts that were rejected
        elif i % 16 == 2:
            change.append(0)
        else:
            change.append(1 + i % 7)  # drafts
    return lens, change


def _grown(case):
    return sum(max(0, c) for c in _changes(case)[1])


# ---- inputs ----------------------------------------------------------------------------------

def _quantise(x):
    """e4m3 codes and the fp32 scale of each row (the last axis)."""
    x = x.float()
    scale = x.abs().amax(-1) / 448.0
    scale = torch.where(scale < TINY, torch.ones_like(scale), scale)
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _pool(case, pages, gen):
    """Keys or values of a pool of pages, logical (pages, page, heads, head_dim), and the scales."""
    heads, dim, page = case["kv_heads"], case["head_dim"], case["page"]
    shape = (pages, heads, page, dim) if case["major"] == "heads" else (pages, page, heads, dim)
    x, scale = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16), None
    if case["cache"] == "e4m3":
        x, scale = _quantise(x)
    else:
        x = x.to(DTYPES[case["cache"]])
    if case["major"] == "heads":
        x = x.transpose(1, 2)
        scale = None if scale is None else scale.transpose(1, 2)
    return x, scale


def _pages(n, page):
    return -(-n // page)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _prepare_resize(case, gen):
    lens, change = _changes(case)
    page, batch = case["page"], case["batch"]
    new = [max(0, n + c) for n, c in zip(lens, change)]
    held = [_pages(n, page) for n in lens]
    taken = sum(max(0, _pages(n, page) - h) for n, h in zip(new, held))
    back = sum(max(0, h - _pages(n, page)) for n, h in zip(new, held))
    cols = max(1, max(max(_pages(n, page), h) for n, h in zip(new, held)) + 3)
    # pages that are free before the call: more than enough, or too few with those that come back
    free = max(0, taken - back - 1 - taken // 3) if case["short"] else taken + 5
    pages = sum(held) + free
    order = torch.randperm(max(1, pages), generator=gen, device="cuda").to(torch.int32)
    table = torch.full((batch, cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(held):
        table[b, :c] = order[at:at + c]
        at += c
    stack = torch.full((max(1, pages),), -1, dtype=torch.int32, device="cuda")
    stack[:free] = order[at:at + free]
    tokens = _grown(case)
    return dict(case=case, op="resize", table=table, lens=_i32(lens), change=_i32(change), free=stack, count=_i32([free]),
                lens_host=lens, change_host=change, free_host=free,
                lens_out=torch.zeros(batch, dtype=torch.int32, device="cuda"), count_out=_i32([0]), missing=_i32([0]),
                starts=torch.zeros(batch + 1, dtype=torch.int32, device="cuda"),
                slots=torch.zeros(tokens + 3, dtype=torch.int64, device="cuda"),
                positions=torch.zeros(tokens + 3, dtype=torch.int32, device="cuda"))


def _prepare_prompt(case, gen):
    dtype, heads, dim, group = DTYPES[case["dtype"]], case["kv_heads"], case["head_dim"], case["q_heads"] // case["kv_heads"]
    n, m = _queries(case), _keys(case)
    tokens, rows = sum(n) + case["pad"], sum(m) + (case["pad"] if n == m else 0)
    if case["fused"] and n == m:  # a projection's rows: queries, keys and values of a token side by side
        x = torch.randn(tokens, (group + 2) * heads * dim, generator=gen, device="cuda", dtype=dtype)
        q, k, v = (y.unflatten(1, (-1, dim)) for y in x.split([group * heads * dim, heads * dim, heads * dim], 1))
        q.mul_(2.5)  # logits of standard deviation 2.5: some rows are sharp, some flat
    else:
        q = (2.5 * torch.randn(tokens, group * heads, dim, generator=gen, device="cuda")).to(dtype)
        k, v = (torch.randn(rows, heads, dim, generator=gen, device="cuda", dtype=dtype) for _ in range(2))
    return dict(case=case, op="prompt", q=q, k=k, v=v, n=n, m=m, starts=_i32(_starts(n)),
                key_starts=None if n == m else _i32(_starts(m)),
                out=torch.zeros(tokens, group * heads, dim, device="cuda", dtype=dtype),
                lse=torch.zeros(tokens, group * heads, device="cuda"))


def _tree_masks(n, rng):
    """Ancestors of the n tokens of a drafted tree, itself among them, as bits of 64-bit words."""
    masks = []
    for i in range(n):
        up = rng.integers(max(-1, i - 6), i) if i else -1
        masks.append((masks[up] if up >= 0 else 0) | 1 << i)
    return [x - (1 << 64) if x >> 63 else x for x in masks]


def _prepare_tree(case, gen, seed):
    dtype, page = DTYPES[case["dtype"]], case["page"]
    n, m = _queries(case), _keys(case)
    need = [_pages(x, page) for x in m]
    pages = max(1, sum(need))
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["batch"], max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    (k, ks), (v, vs) = _pool(case, pages, gen), _pool(case, pages, gen)
    rng = np.random.default_rng(seed)
    masks = None if case["chain"] else [x for c in n for x in _tree_masks(c, rng)]
    q = (2.5 * torch.randn(sum(n), case["q_heads"], case["head_dim"], generator=gen, device="cuda")).to(dtype)
    state = dict(case=case, op="tree", q=q, k=k, v=v, ks=ks, vs=vs, table=table, n=n, m=m, lens=_i32(m), starts=_i32(_starts(n)),
                 max_len=max(m), masks=None if masks is None else torch.tensor(masks, dtype=torch.int64, device="cuda"),
                 out=torch.zeros_like(q), lse=torch.zeros(q.shape[:2], device="cuda"))
    if own:
        import layout_permuting_copy_amd as L
        state["cache"] = L.PagedCache(k, v, ks, vs)
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "resize":
        return _prepare_resize(case, gen)
    return _prepare_prompt(case, gen) if case["op"] == "prompt" else _prepare_tree(case, gen, seed)


# ---- one pass --------------------------------------------------------------------------------

def _plain_resize(s):
    page, batch, cap = s["case"]["page"], s["case"]["batch"], s["free"].numel()
    lens, change = s["lens"].long(), s["change"].long()
    new = (lens + change).clamp(min=0)
    had, has = (lens + page - 1) // page, (new + page - 1) // page
    col = torch.arange(s["table"].shape[1], device="cuda")
    back = (col >= has.unsqueeze(1)) & (col < had.unsqueeze(1))
    pages = s["table"][back]
    top = s["free_host"] + pages.numel()
    s["free"][s["free_host"]:top] = pages
    want = (col >= had.unsqueeze(1)) & (col < has.unsqueeze(1))
    rank = top - want.view(-1).long().cumsum(0).view(want.shape)
    got = torch.where(rank >= 0, s["free"][rank.clamp(0, cap - 1)], torch.full_like(s["table"], -1))
    s["table"].copy_(torch.where(want, got, s["table"]))
    need = want.sum()
    s["missing"][0] = (need - top).clamp(min=0)
    s["count_out"][0] = (top - need).clamp(min=0)
    s["lens_out"].copy_(new)
    grown = (new - lens).clamp(min=0)
    ends = grown.cumsum(0)
    s["starts"][0] = 0
    s["starts"][1:] = ends
    t = torch.arange(s["slots"].numel(), device="cuda")
    b = (t.unsqueeze(1) >= ends.unsqueeze(0)).sum(1)
    real = b < batch
    b = b.clamp(max=batch - 1)
    row = lens[b] + t - (ends - grown)[b]
    row = torch.where(real, row, torch.zeros_like(row))
    at = s["table"][b, row // page].long()
    no = torch.full_like(row, -1)
    s["slots"].copy_(torch.where(real & (at >= 0), at * page + row % page, no))
    s["positions"].copy_(torch.where(real, row, no))


def _resize_outputs(s):
    return [s[x] for x in ("table", "lens_out", "count_out", "missing", "free", "starts", "slots", "positions")]


def _plain_heads(q, k, v, seen, out, lse):
    """Attention of q (n, q_heads, dim) over k, v (m, heads, dim) in 32 bits, `seen` (n, m) or None."""
    dim, heads = q.shape[2], k.shape[1]
    group = q.shape[1] // heads
    for h in range(q.shape[1]):
        kh, vh = k[:, h // group].float(), v[:, h // group].float()
        x = torch.matmul(q[:, h].float(), kh.t().contiguous()) / math.sqrt(dim)
        if seen is not None:
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total == 0, torch.ones_like(total), total)
        out[:, h] = torch.matmul(p, vh).to(out.dtype)
        lse[:, h] = (top + torch.log(total))[:, 0]


def _before(n, m):
    """Which of m rows the last n of them see, causally."""
    return torch.arange(m, device="cuda").unsqueeze(0) <= torch.arange(m - n, m, device="cuda").unsqueeze(1)


def _plain_prompt(s):
    a = c = 0
    for n, m in zip(s["n"], s["m"]):
        if n:
            _plain_heads(s["q"][a:a + n], s["k"][c:c + m], s["v"][c:c + m], _before(n, m) if s["case"]["causal"] else None,
                         s["out"][a:a + n], s["lse"][a:a + n])
        a, c = a + n, c + m


def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _tree_seen(masks, n, m):
    """Which of m rows the last n of them see by the bits of their masks."""
    seen = torch.ones(n, m, dtype=torch.bool, device="cuda")
    seen[:, m - n:] = (masks.unsqueeze(1) >> torch.arange(n, device="cuda").unsqueeze(0)) & 1 == 1
    return seen


def _plain_tree(s):
    a, page = 0, s["case"]["page"]
    for b, (n, m) in enumerate(zip(s["n"], s["m"])):
        if n == 0:
            continue
        i = torch.arange(m, device="cuda")
        pages, rows = s["table"][b][i // page].long(), i % page
        k, v = (_bits(s[x])[pages, rows].view(s[x].dtype).float() for x in ("k", "v"))
        if s["ks"] is not None:
            k, v = k * s["ks"][pages, rows].unsqueeze(-1), v * s["vs"][pages, rows].unsqueeze(-1)
        seen = _before(n, m) if s["masks"] is None else _tree_seen(s["masks"][a:a + n], n, m)
        _plain_heads(s["q"][a:a + n], k, v, seen, s["out"][a:a + n], s["lse"][a:a + n])
        a += n


def run(state):
    s = state
    if own:
        import layout_permuting_copy_amd as L
    if s["op"] == "resize":
        if own:
            L.tc_paged_resize(s["table"], s["lens"], s["change"], s["free"], s["count"], s["case"]["page"],
                              lens_out=s["lens_out"], count_out=s["count_out"], token_starts=s["starts"], slots=s["slots"],
                              positions=s["positions"], missing=s["missing"])
        else:
            _plain_resize(s)
        return _resize_outputs(s)
    if s["op"] == "prompt":
        if own:
            L.tc_prompt_attention(s["q"], s["k"], s["v"], s["starts"], key_starts=s["key_starts"], causal=s["case"]["causal"],
                                  out=s["out"], lse=s["lse"])
        else:
            _plain_prompt(s)
    elif own:
        L.tc_paged_tree_attention(s["q"], s["cache"], s["table"], s["lens"], s["starts"], masks=s["masks"],
                                  max_len=s["max_len"], out=s["out"], lse=s["lse"])
    else:
        _plain_tree(s)
    return [s["out"], s["lse"]]


# ---- the definitions in 64 bits --------------------------------------------------------------

def _exact_resize(s):
    page = s["case"]["page"]
    table, stack = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    free = list(stack[:s["free_host"]])
    lens, starts, missing = [], [0], 0
    for b, (n, c) in enumerate(zip(s["lens_host"], s["change_host"])):
        new = max(0, n + c)
        lens.append(new)
        starts.append(starts[-1] + max(0, new - n))
        for i in range(_pages(new, page), _pages(n, page)):
            free.append(table[b, i])
    stack[:len(free)] = free
    for b, (n, new) in enumerate(zip(s["lens_host"], lens)):
        for i in range(_pages(n, page), _pages(new, page)):
            missing += not free
            table[b, i] = free.pop() if free else -1
    slots = np.full(s["slots"].numel(), -1, dtype=np.int64)
    positions = np.full(s["slots"].numel(), -1, dtype=np.int32)
    for b, (n, new) in enumerate(zip(s["lens_host"], lens)):
        rows = np.arange(n, max(n, new))
        at = table[b, rows // page].astype(np.int64)
        slots[starts[b]:starts[b + 1]] = np.where(at >= 0, at * page + rows % page, -1)
        positions[starts[b]:starts[b + 1]] = rows
    i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()
    return [i32(table), i32(lens), i32([len(free)]), i32([missing]), i32(stack), i32(starts), torch.from_numpy(slots).cuda(),
            i32(positions)]


def _exact_sequence(q, k, v, visible, out, lse):
    """One sequence by its definition, query head by query head and 4096 queries at a time."""
    group = q.shape[1] // k.shape[1]
    for h in range(k.shape[1]):
        keys, values = k[:, h].double(), v[:, h].double()
        for g in range(h * group, (h + 1) * group):
            for i in range(0, q.shape[0], 4096):
                x = (keys @ q[i:i + 4096, g].double().T).T.mul_(q.shape[2] ** -0.5)
                hidden = visible(i, x.shape[0])
                if hidden is not None:
                    x.masked_fill_(hidden, -math.inf)
                total = torch.logsumexp(x, 1)
                p = x.sub_(total.masked_fill(total == -math.inf, 0.0)[:, None]).exp_()
                out[i:i + 4096, g] = p @ values
                lse[i:i + 4096, g] = total


def _exact_attention(case, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    a = c = 0
    table = None if case["op"] == "prompt" else s["table"].cpu().numpy()
    for b, (n, m) in enumerate(zip(s["n"], s["m"])):
        first = m - n
        if case["op"] == "prompt":
            k, v = s["k"][c:c + m], s["v"][c:c + m]
        elif n:
            at = np.arange(m)
            page, row = (torch.from_numpy(x).cuda() for x in (table[b][at // case["page"]].astype(np.int64), at % case["page"]))
            k, v = (_bits(s[x])[page, row].view(s[x].dtype).float().double() for x in ("k", "v"))
            if s["ks"] is not None:
                k, v = (x * y[page, row].double()[..., None] for x, y in ((k, s["ks"]), (v, s["vs"])))
        column = torch.arange(m, device="cuda")

        def visible(i, count):
            """What queries i .. i + count - 1 do not see."""
            if case["op"] == "prompt" and not case["causal"]:
                return None
            own_row = first + i + torch.arange(count, device="cuda")
            if case["op"] == "prompt" or s["masks"] is None:
                return column[None, :] > own_row[:, None]
            words = s["masks"][a + i:a + i + count].cpu().numpy().view(np.uint64)
            hidden = np.zeros((count, m), dtype=bool)
            for j in range(n):
                hidden[:, first + j] = (words >> np.uint64(j)) & np.uint64(1) == 0
            return torch.from_numpy(hidden).cuda()

        if n:
            _exact_sequence(s["q"][a:a + n], k, v, visible, out[a:a + n], lse[a:a + n])
        a, c = a + n, c + m
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_resize(s) if case["op"] == "resize" else _exact_attention(case, s)


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    if case["op"] == "resize":
        lens, change = _changes(case)
        moved = sum(abs(_pages(max(0, n + c), case["page"]) - _pages(n, case["page"])) for n, c in zip(lens, change))
        # lengths and changes read, lengths and starts written, pages read and written, slots and positions written
        return {"bytes": 16 * case["batch"] + 8 * moved + 12 * (_grown(case) + 3) + 16, "flops": 0}
    n, m, dim = _queries(case), _keys(case), case["head_dim"]
    causal = case["op"] == "tree" or case["causal"]
    pairs = sum(a * c - (a * (a - 1) // 2 if causal else 0) for a, c in zip(n, m))
    small = sum(n) * case["q_heads"] * (2 * 2 * dim + 4)
    if case["op"] == "prompt":
        rows = sum(m) * case["kv_heads"] * 2 * 2 * dim
    else:
        row = 2 * case["kv_heads"] * (dim + 4 if case["cache"] == "e4m3" else 2 * dim)
        rows = sum((c * row + 4 * _pages(c, case["page"])) for a, c in zip(n, m) if a) + (0 if case["chain"] else 8 * sum(n))
    return {"bytes": rows + small + 4 * len(n), "flops": 4 * pairs * case["q_heads"] * dim}
