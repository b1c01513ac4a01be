"""dsa_paged_slots against a token-by-token walk: every output is a whole number and has to be equal."""
import random

import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(B, page, ctx, new, seed, spare=3):
    r = random.Random(seed)
    lens = [r.choice([0, r.randint(0, ctx), page * r.randint(0, max(0, ctx // page))]) for _ in range(B)]
    news = [r.choice([0, 1, r.randint(0, new)]) for _ in range(B)]
    width = max([-(-(s + n) // page) for s, n in zip(lens, news)] + [1]) + 2
    ids = list(range(B * width + spare + 5))
    r.shuffle(ids)
    table = [[ids.pop() if c < -(-s // page) else -7 for c in range(width)] for s in lens]
    fresh = sum(-(-(s + n) // page) - -(-s // page) for s, n in zip(lens, news))
    free = [ids.pop() if ids else 900000 + i for i in range(fresh + spare)]
    return lens, news, table, free


@pytest.mark.parametrize("B,page,ctx,new", [(1, 1, 5, 3), (3, 16, 100, 40), (7, 33, 200, 1), (300, 64, 900, 5),
                                            (257, 7, 50, 700), (2049, 64, 3000, 9), (8192, 128, 4000, 2)])
@pytest.mark.parametrize("pad", [0, 37])
def test_slots_match_the_walk(B, page, ctx, new, pad):
    lens, news, table, free = make(B, page, ctx, new, seed=B + page)
    N = sum(news) + pad
    want = ref.slots(lens, news, table, free, page, N)
    t = dev(table)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    for _ in range(2):  # the call can be made again: it gives the same answer
        slots, pos, cu, out_lens, taken = dsa.dsa_paged_slots(dev(lens), t, dev(free), page, dev(news), N, ws)
        assert slots.tolist() == want[0] and pos.tolist() == want[1] and cu.tolist() == want[2]
        assert out_lens.tolist() == want[3] and taken.tolist() == [want[4]] and t.tolist() == want[5]
    assert dsa.dsa_read_device_status(ws) == 0


def test_one_token_each_and_an_empty_batch():
    lens, _, table, free = make(40, 16, 90, 1, seed=9)
    want = ref.slots(lens, None, table, free + list(range(5000, 5100)), 16, 40)
    t = dev(table)
    slots, pos, cu, out_lens, taken = dsa.dsa_paged_slots(dev(lens), t, dev(free + list(range(5000, 5100))), 16)
    assert slots.tolist() == want[0] and pos.tolist() == want[1] and t.tolist() == want[5]
    e = dev([])
    slots, pos, cu, out_lens, taken = dsa.dsa_paged_slots(e, torch.empty(0, 4, dtype=torch.int32, device=DEV), e, 16,
                                                          new_lens=e, N=3)
    assert slots.tolist() == [-1] * 3 and pos.tolist() == [-1] * 3 and cu.tolist() == [0] and taken.tolist() == [0]


@pytest.mark.parametrize("why", ["free", "table", "tokens", "negative", "wrap"])
def test_a_step_that_does_not_fit_changes_nothing(why):
    page, lens, news = 16, [10, 16, 40], [3, 17, 1]
    table = [[5, -1, -1], [6, -1, -1], [7, 8, 9]]
    free, N = [20, 21], 21
    if why == "free":
        free = free[:1]
    if why == "table":
        news = [3, 40, 1]
        free, N = list(range(20, 40)), 64
    if why == "tokens":
        N = 20
    if why == "negative":
        news = [3, -1, 1]
    if why == "wrap":
        news = [2 ** 31 - 1, 2 ** 31 - 1, 2]
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    t = dev(table)
    slots, pos, cu, out_lens, taken = dsa.dsa_paged_slots(dev(lens), t, dev(free), page, dev(news), N, ws)
    assert slots.tolist() == [-1] * N and pos.tolist() == [-1] * N and cu.tolist() == [0] * 4
    assert out_lens.tolist() == lens and taken.tolist() == [0] and t.tolist() == table
    assert dsa.dsa_read_device_status(ws) == 8
    assert dsa.dsa_read_device_status(ws) == 0  # read and cleared


def test_a_bad_page_and_rows_past_31_bits_are_reported():
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    slots, pos, *_ = dsa.dsa_paged_slots(dev([5, 5]), dev([[-3], [2]]), dev([]), 16, workspace=ws)
    assert slots.tolist() == [-1, 2 * 16 + 5] and pos.tolist() == [5, 5]
    assert dsa.dsa_read_device_status(ws) == 6
    slots, *_ = dsa.dsa_paged_slots(dev([5, 5]), dev([[2 ** 27], [2 ** 27 - 1]]), dev([]), 16, workspace=ws)
    assert slots.tolist() == [-1, (2 ** 27 - 1) * 16 + 5]
    assert dsa.dsa_read_device_status(ws) == 6


def test_a_captured_step_follows_the_lengths():
    page = 4
    lens, table, free = dev([3, 0]), torch.full((2, 8), -1, dtype=torch.int32, device=DEV), dev(list(range(50, 70)))
    table[0, 0] = 11
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_slots(lens, table.clone(), free, page, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        slots, pos, cu, out_lens, taken = dsa.dsa_paged_slots(lens, table, free, page, workspace=ws)
    got, host = [], [[11], []]
    used, n = 0, [3, 0]
    for _ in range(6):
        g.replay()
        got = slots.tolist()
        for b in range(2):
            if n[b] % page == 0:
                host[b].append(50 + used)
                used += 1
            assert got[b] == host[b][-1] * page + n[b] % page
            n[b] += 1
        lens.copy_(out_lens)
        free.copy_(torch.roll(free, -int(taken)))
    assert lens.tolist() == n and dsa.dsa_read_device_status(ws) == 0
