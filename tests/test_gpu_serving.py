"""A serving loop's operators run together: prompts taken in, chunks of prompts, decoding, drafted trees, rejected drafts,
sequences that leave, every step's attention against the definition on the cache as it stands."""

import math

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


class Loop:
    """The device state of a loop, and the same rows held plainly on the host."""

    def __init__(self, kind, cache_kind, heads, group, dim, page, batch, cols, pages):
        self.gen = torch.Generator().manual_seed(17)
        self.dt, self.cache_kind, self.shape = P.DT[kind], cache_kind, (heads, group, dim)
        pool = P.Pool(cache_kind, pages, page, heads, dim, "heads", fill=0.0)
        self.cache, self.page, self.pages, self.batch = pool.on_gpu(), page, pages, batch
        self.table = torch.full((batch, cols), -1, dtype=torch.int32, device="cuda")
        self.lens, self.count = _i32([0] * batch), _i32([pages])
        self.free = torch.randperm(pages, generator=self.gen).to(torch.int32).cuda()
        self.rows = [[torch.zeros(0, heads, dim)] * 2 for _ in range(batch)]  # keys, values of each sequence

    def held(self):
        return [k.shape[0] for k, _ in self.rows]

    def resize(self, change):
        tokens = sum(max(0, c) for c in change)
        self.starts = _i32([0] * (self.batch + 1))
        slots, positions = torch.zeros(tokens, dtype=torch.int64, device="cuda"), _i32([0] * tokens)
        missing = _i32([-1])
        before = self.held()
        L.tc_paged_resize(self.table, self.lens, _i32(change), self.free, self.count, self.page, token_starts=self.starts, slots=slots,
                          positions=positions, missing=missing)
        assert missing.item() == 0
        assert self.lens.tolist() == [n + c for n, c in zip(before, change)]
        assert positions.tolist() == [n + i for n, c in zip(before, change) for i in range(c)]
        assert slots.unique().numel() == tokens and bool((slots >= 0).all())
        # every page is free or held by one sequence
        held = [self.table[b, :-(-n // self.page)] for b, n in enumerate(self.lens.tolist())]
        all_pages = torch.cat(held + [self.free[:self.count.item()]])
        assert all_pages.sort().values.tolist() == list(range(self.pages))
        for b, c in enumerate(change):
            if c < 0:
                self.rows[b] = [x[:x.shape[0] + c] for x in self.rows[b]]
        return slots

    def append(self, change, slots):
        heads, group, dim = self.shape
        tokens = sum(max(0, c) for c in change)
        q = (2.0 * torch.randn(tokens, heads * group, dim, generator=self.gen)).to(self.dt)
        k, v = (torch.randn(tokens, heads, dim, generator=self.gen).to(self.dt) for _ in range(2))
        L.tc_paged_append(self.cache, k.cuda(), v.cuda(), self.table, self.lens, token_starts=self.starts)
        held = []
        for x, new in ((self.cache.k, k), (self.cache.v, v)):
            s = self.cache.k_scale if x is self.cache.k else self.cache.v_scale
            # the rows lie where the slots say
            got = P.bits(x)[slots // self.page, slots % self.page].view(x.dtype).float()
            if s is None:
                assert torch.equal(got.cpu(), new.float())
            else:
                got = got * s[slots // self.page, slots % self.page].unsqueeze(-1)
            held.append(got.double().cpu())
        at = 0
        for b, c in enumerate(change):
            if c > 0:
                self.rows[b] = [torch.cat([x.double(), y[at:at + c]]) for x, y in zip(self.rows[b], held)]
                at += c
        return q, k, v

    def want(self, q, change, seen_of):
        kind = torch.bfloat16 if self.cache_kind == "e4m3" else self.dt
        parts, at = [], 0
        for b, c in enumerate(change):
            if c > 0:
                k, v = self.rows[b]
                parts.append(R.sequence(q[at:at + c], k, v, seen_of(at, c, k.shape[0]), None, R.half_step(kind)))
                at += c
        ref = [torch.cat(p) for p in zip(*parts)]
        ref[2] += 2.0 ** -32 * 5.0 * 1000  # fp16's subnormal weights: 2^-32 of the greatest, for up to 1000 values
        return ref

    def check(self, out, lse, ref, what):
        say(f"[gpu] {what}")
        R.close(out, ref[0], ref[2], what, self.dt)
        R.close(lse, ref[1], ref[3], what + ", lse")

    def tree(self, q, masks=None):
        lse = torch.zeros(q.shape[:2], device="cuda")
        out = L.tc_paged_tree_attention(q.cuda(), self.cache, self.table, self.lens, self.starts,
                                        masks=None if masks is None else torch.tensor(masks, device="cuda"), lse=lse)
        return out, lse


@pytest.mark.parametrize("kind, cache_kind", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
def test_a_serving_loop(kind, cache_kind):
    batch, page = 4, 16
    s = Loop(kind, cache_kind, 2, 4, 64, page, batch, 40, 100)
    before = lambda at, n, m: R.before(n, m)

    def prompts(change):
        slots = s.resize(change)
        q, k, v = s.append(change, slots)
        lse = torch.zeros(q.shape[:2], device="cuda")
        out = L.tc_prompt_attention(q.cuda(), k.cuda(), v.cuda(), s.starts, lse=lse)
        if cache_kind != "e4m3":
            s.check(out, lse, s.want(q, change, before), f"prompts {change}")
        out, lse = s.tree(q)
        s.check(out, lse, s.want(q, change, before), f"prompts over the cache {change}")

    def chunk(change):
        q, _, _ = s.append(change, s.resize(change))
        out, lse = s.tree(q)
        s.check(out, lse, s.want(q, change, before), f"chunks {change}")

    def decode():
        change = [1] * batch
        q, _, _ = s.append(change, s.resize(change))
        lse = torch.zeros(q.shape[:2], device="cuda")
        out = L.tc_paged_attention(q.cuda(), s.cache, s.table, s.lens, lse=lse)
        s.check(out, lse, s.want(q, change, before), "a step")

    def draft(sizes, accepted):
        """Trees whose first branch is a chain; `accepted` of its tokens stay."""
        masks = []
        for n, keep in zip(sizes, accepted):
            words = []
            for i in range(n):
                up = i - 1 if i < keep else int(torch.randint(0, i, (1,), generator=s.gen)) if i else -1
                words.append((words[up] if up >= 0 else 0) | 1 << i)
            masks += words
        q, _, _ = s.append(sizes, s.resize(sizes))
        out, lse = s.tree(q, masks)
        s.check(out, lse, s.want(q, sizes, lambda at, n, m: R.by_masks(masks[at:at + n], n, m)), f"drafts {sizes}")
        s.resize([a - n for n, a in zip(sizes, accepted)])

    prompts([130, 40, 7, 1])
    decode()
    draft([12, 30, 1, 62], [5, 0, 1, 17])
    chunk([64, 0, 200, 3])
    draft([8, 8, 8, 8], [8, 1, 0, 3])
    decode()
    s.resize([-s.held()[0], 0, -s.held()[2], 0])
    s.resize([0, 0, 0, 0])
    prompts([500, 0, 33, 0])
    decode()
    s.resize([-n for n in s.held()])
    assert s.count.item() == s.pages


def test_a_prompt_in_pieces_is_the_prompt():
    """Chunks over the cache give what one packed call does, up to how their sums are dealt out."""
    s = Loop("bf16", "bf16", 2, 2, 128, 16, 1, 64, 64)
    heads, group, dim = s.shape
    n, cuts = 700, [0, 1, 90, 500, 700]
    q = torch.randn(n, heads * group, dim, generator=s.gen).to(torch.bfloat16).cuda()
    k, v = (torch.randn(n, heads, dim, generator=s.gen).to(torch.bfloat16).cuda() for _ in range(2))
    whole = L.tc_prompt_attention(q, k, v, _i32([0, n]))
    ref = R.sequence(q.cpu(), k.cpu(), v.cpu(), R.before(n, n))
    for a, b in zip(cuts, cuts[1:]):
        s.rows[0] = [torch.zeros(a, heads, dim)] * 2
        s.resize([b - a])
        L.tc_paged_append(s.cache, k[a:b], v[a:b], s.table, s.lens, token_starts=s.starts)
        out = L.tc_paged_tree_attention(q[a:b], s.cache, s.table, s.lens, s.starts)
        R.close(out, ref[0][a:b], ref[2][a:b], "out", torch.bfloat16)
        R.close(out, whole[a:b].cpu().double(), 2 * (ref[2][a:b] + 2.0 ** -8 * ref[0][a:b].abs()), "beside the whole")
    assert math.isfinite(float(out.float().sum()))
