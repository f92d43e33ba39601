"""Block tables that grow and shrink on the GPU, against the definition."""

import random

import pytest
import torch

import layout_permuting_copy_amd as L
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


def _check(table, lens, change, stack, count, page, tokens, in_place=False, table_d=None):
    want = R.resize(table, lens, change, stack, count, page, tokens)
    t = _i32(table) if table_d is None else table_d
    n, c, s, k = _i32(lens), _i32(change), _i32(stack), _i32([count])
    n_out, k_out = (n, k) if in_place else (_i32([-7] * len(lens)), _i32([-7]))
    starts, missing = _i32([-7] * (len(lens) + 1)), _i32([-7])
    slots = torch.full((tokens,), -7, dtype=torch.int64, device="cuda")
    positions = _i32([-7] * tokens)
    got = L.tc_paged_resize(t, n, c, s, k, page, lens_out=n_out, count_out=k_out, token_starts=starts, slots=slots,
                            positions=positions, missing=missing)
    assert got is n_out
    for name, x, y in zip(("table", "lens", "stack", "count", "missing", "starts", "slots", "positions"),
                          (t, n_out, s, k_out, missing, starts, slots, positions),
                          want):
        y = [y] if isinstance(y, int) else y
        assert x.tolist() == y, name
    if not in_place:
        assert n.tolist() == lens and k.tolist() == [count] and c.tolist() == change
    return want


def _case(rng, batch, page, longest, mix, short=False):
    lens, change = [], []
    for _ in range(batch):
        n = rng.randint(0, longest)
        lens.append(n)
        change.append({"grow": lambda: rng.randint(0, longest), "step": lambda: 1, "gone": lambda: -n,
                       "mixed": lambda: rng.choice([0, 1, -n, -n - 3, -rng.randint(0, n), rng.randint(0, 2 * longest)])}[mix]())
    pages = lambda n: -(-n // page)
    cols = max([1] + [pages(max(n, n + c)) for n, c in zip(lens, change)]) + 1
    held = [pages(n) for n in lens]
    need = sum(max(0, pages(max(0, n + c)) - h) for n, c, h in zip(lens, change, held))
    free = need // 3 if short else need + 2
    order = list(range(sum(held) + free))
    rng.shuffle(order)
    table, at = [], 0
    for h in held:
        table.append(order[at:at + h] + [-9] * (cols - h))
        at += h
    return table, lens, change, order[at:] + [-9] * (len(order) - free), free


@pytest.mark.parametrize("batch, page, longest", [(1, 16, 40), (3, 1, 9), (48, 16, 700), (65, 7, 100), (300, 64, 500), (1023, 16, 40),
                                                  (1024, 16, 3), (1025, 24, 60), (2500, 5, 33)])
@pytest.mark.parametrize("mix", ["grow", "step", "gone", "mixed"])
@pytest.mark.parametrize("short", [False, True])
def test_resize(batch, page, longest, mix, short):
    rng = random.Random(f"{batch} {page} {longest} {mix} {short}")
    table, lens, change, stack, free = _case(rng, batch, page, longest, mix, short)
    total = sum(max(0, c) for c in change)
    say(f"[gpu] {total} new rows")
    for tokens in (total + 5, total // 2):
        _check(table, lens, change, stack, free, page, tokens, in_place=tokens == total // 2)


def test_resize_of_long_prompts():
    """More new rows than one workgroup places, a sequence of one beside them, pages of one row."""
    for lens, change, page in (([0, 5, 100], [20000, 1, 9000], 16), ([3] * 9, [4000] * 9, 1), ([17], [8192], 32), ([17], [8193], 32)):
        cols = max(-(-(n + c) // page) for n, c in zip(lens, change))
        held = [-(-n // page) for n in lens]
        need = sum(-(-(n + c) // page) for n, c in zip(lens, change)) + 3
        order = list(range(need))
        random.Random(1).shuffle(order)
        table, at = [], 0
        for h in held:
            table.append(order[at:at + h] + [-1] * (cols - h))
            at += h
        say(f"[gpu] {sum(change)} new rows in pages of {page}")
        _check(table, lens, change, order[at:] + [-1] * at, need - at, page, sum(change) + 1000)


def test_resize_at_the_edges():
    most = 2 ** 31 - 1
    # lengths below zero count as none, the table's columns bound the pages, sums stop at 2^31 - 1
    _check([[4, 5, -1], [6, -1, -1]], [-5, 16], [17, most], [0, 1, 2, 3, 7, 8], 6, 16, 40)
    _check([[0], [1]], [most, most], [5, 5], [3, 4], 2, 16, 4)
    # shrinking by more than there is; entries that are no pages; a stack without room, and one that counts too many
    _check([[3, -1, 5], [7, 8, 9]], [48, 48], [-100, -17], [0, 1, 2, -1, -1], 3, 16, 4)
    _check([[3, 4, 5]], [48], [-48], [0, 1, 2, 6], 3, 16, 0)
    _check([[-1, -1, -1]], [0], [40], [0, 1, 2, 6], 9, 16, 40)
    _check([[-1, -1, -1]], [0], [40], [0, 1, 2, 6], -2, 16, 40)
    # pages that come back are handed out in the same call
    _check([[3, 4], [-1, -1]], [32, 0], [-32, 32], [-1, -1], 0, 16, 32)
    _check([[3, 4], [-1, -1]], [0, 32], [16, -32], [], 0, 16, 16)
    # no sequences, no columns
    starts, count = _i32([-7]), _i32([9])
    slots = torch.full((3,), -7, dtype=torch.int64, device="cuda")
    e = _i32([])
    L.tc_paged_resize(_i32([]).view(0, 4), e, e, _i32([1, 2, 3]), count, 16, token_starts=starts, slots=slots)
    assert starts.tolist() == [0] and slots.tolist() == [-1] * 3 and count.tolist() == [3]
    n = _i32([5, 0])
    L.tc_paged_resize(_i32([]).view(2, 0), n, _i32([3, 2]), _i32([1, 2, 3]), count, 16, token_starts=_i32([0] * 3), slots=slots)
    assert n.tolist() == [8, 2] and slots.tolist() == [-1] * 3 and count.tolist() == [3]


@pytest.mark.parametrize("tokens", [64, 8192, 8193, 20000])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_of_the_sequence_past_which_the_starts_stop(tokens, in_place):
    """A sequence whose end the starts no longer count has its rows counted from its own first, also where its old length
    cannot be had from its new one."""
    most = 2 ** 31 - 1
    for lens, change in (([0, 0], [5000, most]), ([0, 7], [10, most]), ([33, 100, 4], [-33, most - 99, 9]), ([5, 0, 40, 3], [0, 17, most, most]),
                         ([2], [most - 2]), ([2], [most]), ([0] * 1500 + [21, 6], [3] * 1500 + [most - 5000, 9]),
                         ([most - 3, 0], [3, most - 3]), ([9] * 1025, [0] * 1024 + [most])):
        held = [min(-(-n // 16), 700) for n in lens]
        order = list(range(sum(held) + 900))
        random.Random(len(lens)).shuffle(order)
        table, at = [], 0
        for h in held:
            table.append(order[at:at + h] + [-1] * (700 - h))
            at += h
        say(f"[gpu] {lens[:4]} + {change[:4]}, {tokens} places")
        _check(table, lens, change, order[at:] + [-1] * at, 900, 16, tokens, in_place=in_place)


def test_resize_of_a_strided_table_without_the_rows_places():
    rng = random.Random(5)
    table, lens, change, stack, free = _case(rng, 40, 16, 200, "mixed")
    want = R.resize(table, lens, change, stack, free, 16, 0)
    wide = torch.full((len(table[0]), 2 * len(table)), -3, dtype=torch.int32, device="cuda")
    t = wide.t()[::2]
    t.copy_(_i32(table))
    n, k, s = _i32(lens), _i32([free]), _i32(stack)
    L.tc_paged_resize(t, n, _i32(change), s, k, 16)
    assert t.tolist() == want[0] and n.tolist() == want[1] and s.tolist() == want[2] and k.tolist() == [want[3]]
    assert bool((wide.t()[1::2] == -3).all())
    positions, starts = _i32([-7] * 4), _i32([0] * 41)
    L.tc_paged_resize(t, n, _i32([0] * 39 + [2]), s, k, 16, token_starts=starts, positions=positions)
    assert positions.tolist() == [want[1][39], want[1][39] + 1, -1, -1]


@pytest.mark.parametrize("tokens", [64, 9000])
def test_a_captured_resize_replays_in_place(tokens):
    """Lengths, table and stack move on from replay to replay, with the program's own work between them."""
    rng = random.Random(tokens)
    batch, page, cols = 5, 16, 200
    table, stack, count, lens = [[-1] * cols for _ in range(batch)], list(range(batch * cols)), batch * cols, [0] * batch
    rng.shuffle(stack)
    t, n, s, k, c = _i32(table), _i32(lens), _i32(stack), _i32([count]), _i32([0] * batch)
    starts, positions = _i32([0] * (batch + 1)), _i32([0] * tokens)
    slots = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        L.tc_paged_resize(t, n, c, s, k, page, token_starts=starts, slots=slots, positions=positions)
    for step in range(6):
        change = [rng.choice([1, 0, -rng.randint(0, 40), rng.randint(0, 500), -m]) for m in lens]
        c.copy_(_i32(change))
        (torch.randn(1 << 18, device="cuda") * 2).sum().item()
        table, lens, stack, count, _, want_starts, want_slots, want_positions = R.resize(table, lens, change, stack, count, page, tokens)
        g.replay()
        torch.cuda.synchronize()
        say(f"[gpu] replay {step}")
        assert n.tolist() == lens and k.tolist() == [count] and t.tolist() == table and s.tolist() == stack
        assert starts.tolist() == want_starts and slots.tolist() == want_slots and positions.tolist() == want_positions
