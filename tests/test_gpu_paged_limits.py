"""The serving calls at their largest sizes, two at a time, and with a workspace that two graphs share."""
import math

import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def dev(v):
    return torch.tensor(v, dtype=I32, device=DEV)


def test_slots_of_the_most_tokens():
    # N = 2^31 - 1 entries, of which two are tokens: every other one is -1
    N = 2 ** 31 - 1
    table = torch.full((2, 4), -1, dtype=I32, device=DEV)
    slots, pos, cu, lens, taken = dsa.dsa_paged_slots(dev([5, 0]), table, dev([3, 1, 2]), 16, new_lens=dev([0, 2]), N=N)
    assert slots[:2].tolist() == [48, 49] and pos[:2].tolist() == [0, 1] and int(taken) == 1 and table[1, 0] == 3
    for t in (slots, pos):
        assert bool((t[2:] == -1).all())
        del t
    del slots, pos
    torch.cuda.empty_cache()


@pytest.mark.parametrize("D", [1, 8])
def test_rows_up_to_the_last_count(D):
    # one row, read by a stride of zero, on every row of an output past 2^31 elements
    T = 2 ** 31 - 65
    one = torch.arange(1, D + 1, dtype=torch.bfloat16, device=DEV)
    out = dsa.dsa_norm_rope_fwd(one.expand(T, D))
    words = out.view(-1) if D == 1 else out.view(torch.int64).view(-1, 2)
    for part in words.split(2 ** 28):
        assert bool((part == (one if D == 1 else one.view(torch.int64))).all())
    del out, words, part
    torch.cuda.empty_cache()


def test_a_request_of_the_longest_length():
    # 2^31 - 1 positions in one page of 64 that the table names again and again.  Every CTA adds its 2^25 / 152 tiles one
    # after the other: sums of positive terms, each addition off by at most 2^-24 of the sum.
    g = torch.Generator().manual_seed(5)
    cache = torch.randn(1, 64, 512, generator=g).bfloat16()
    q = torch.randn(1, 1, 512, generator=g).bfloat16()
    table = torch.zeros(1, 2 ** 25, dtype=I32, device=DEV)
    ws = torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV)
    out, lse = dsa.dsa_paged_mla(q.to(DEV), cache.to(DEV), table, dev([2 ** 31 - 1]), 0.04, workspace=ws)
    z = 0.04 * (cache[0].double() @ q[0, 0].double())
    want = math.log(2.0 ** 25) + float(torch.logsumexp(z, 0))
    assert abs(float(lse) - want) <= 2 ** 25 / 152 * 2.0 ** -24 + 2.0 ** -12
    assert bool(torch.isfinite(out).all()) and dsa.dsa_read_device_status(ws) == 0


def step_inputs(seed, B=5, H=64, L=900, page=16, Hi=16):
    g = torch.Generator().manual_seed(seed)
    lens = [L - 37 * b for b in range(B)]
    need = -(-L // page)
    pages = torch.randperm(B * need, generator=g).view(B, need)
    return dict(q=torch.randn(B, H, 576, generator=g).bfloat16().to(DEV),
                cache=torch.randn(B * need, page, 576, generator=g).bfloat16().to(DEV), table=pages.to(I32).to(DEV),
                lens=dev(lens), qi=torch.randn(B, Hi, 128, generator=g).bfloat16().to(DEV),
                keys=torch.randn(B * need, page, 128, generator=g).bfloat16().to(DEV),
                w=torch.randn(B, Hi, generator=g).to(DEV))


def attend(s, ws, wt):
    idx, n = dsa.dsa_paged_indexer_topk(s["qi"], s["keys"], s["w"], s["table"], s["lens"], 100, max_len=1024, workspace=wt)
    out, lse = dsa.dsa_paged_mla(s["q"], s["cache"], s["table"], s["lens"], 0.04, topk_idx=idx, topk_len=n, workspace=ws)
    full, _ = dsa.dsa_paged_mla(s["q"], s["cache"], s["table"], s["lens"], 0.04, workspace=ws)
    return idx, n, out, lse, full


def spaces():
    return (torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV),
            torch.zeros(dsa.paged_workspace_size("topk", 5, 1024), dtype=torch.uint8, device=DEV))


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_calls_at_once():
    # two streams, each with its own workspaces, many calls in flight: the bits of one call after the other
    sets = [step_inputs(s) for s in (1, 2)]
    want = [attend(s, *spaces()) for s in sets]
    torch.cuda.synchronize()
    streams, own = [torch.cuda.Stream() for _ in sets], [spaces() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(attend(sets[k], *own[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(equal(x, want[k]) for x in got[k])
        assert all(dsa.dsa_read_device_status(w) == 0 for w in own[k])


@pytest.mark.parametrize("lists", [False, True])
def test_thousands_of_short_requests(lists):
    # 20 and more groups of one or two tiles for every CTA, so that many end and open one, or lie between two ends
    B, H, page = 3200, 3, 8
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(0, 90, (B,), generator=g)
    need = [-(-int(n) // page) for n in lens]
    pool = 400  # pages that the requests share
    table = torch.full((B, 12), -1, dtype=I32)
    for b, k in enumerate(need):
        table[b, :k] = torch.randint(0, pool, (k,), generator=g, dtype=I32)
    cache = torch.randn(pool, page, 576, generator=g).bfloat16()
    q = torch.randn(B, H, 576, generator=g).bfloat16()
    idx = None
    if lists:
        idx = (torch.rand(B, 6, generator=g) * lens.clamp(min=1)[:, None]).to(I32)
        idx[lens == 0] = -1
    ws = spaces()[0]
    out, lse = dsa.dsa_paged_mla(q.to(DEV), cache.to(DEV), table.to(DEV), lens.to(I32).to(DEV), 0.04, workspace=ws,
                                 topk_idx=None if idx is None else idx.to(DEV))
    want, want_lse = ref.paged_mla(q, cache, table.tolist(), lens.tolist(), list(range(B + 1)), 0.04, page, None, idx)
    out, lse = out.cpu().double(), lse.cpu().double()
    # half a bf16 step for the rounding; scores in fp32 and weights as hi + lo: 2^-13 of the largest value
    assert bool(((out - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -13 * 5.0).all())
    seen = ~torch.isinf(want_lse)
    assert torch.equal(seen, ~torch.isinf(lse)) and bool(((lse - want_lse)[seen].abs() <= 2.0 ** -13).all())
    assert dsa.dsa_read_device_status(ws) == 0


def test_two_graphs_share_a_workspace():
    sets = [step_inputs(s) for s in (3, 4)]
    ws, wt = spaces()
    want = [attend(s, *spaces()) for s in sets]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(attend(s, ws, wt))
        graphs.append(g)
    for k in (0, 1, 1, 0, 1, 0):
        for t in got[k]:
            t.zero_()
        graphs[k].replay()
        assert equal(got[k], want[k])
    assert dsa.dsa_read_device_status(ws) == 0 and dsa.dsa_read_device_status(wt) == 0


def test_a_position_named_twice_counts_twice():
    # a list of [5, 5, 9]: the weights of the formula with position 5 counted twice
    s = step_inputs(6, B=1, H=16, L=40)
    out, lse = dsa.dsa_paged_mla(s["q"], s["cache"], s["table"], s["lens"], 0.04, topk_idx=dev([[5, 5, 9]]))
    rows = s["cache"].view(-1, 576)[ref.rows_of(s["table"][0].tolist(), [5, 5, 9], 16)].double()
    z = 0.04 * s["q"][0].double() @ rows.T
    want = torch.softmax(z, 1) @ rows[:, :512]
    # half a bf16 step for the rounding; scores in fp32 and weights as hi + lo: 2^-13 of the largest value
    assert bool(((out[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -13 * rows.abs().max()).all())
    assert bool(((lse[0].double() - torch.logsumexp(z, 1)).abs() <= 2.0 ** -13).all())


def test_backwards_at_once_and_in_one_graph():
    # the sums of two gradients in flight, eager on two streams and captured one after the other with one workspace
    g = torch.Generator().manual_seed(9)
    sets = [(torch.randn(5000, 128, generator=g).bfloat16().to(DEV), torch.randn(5000, 128, generator=g).bfloat16().to(DEV),
             torch.randn(128, generator=g).to(DEV)) for _ in range(2)]
    make = lambda: torch.zeros(dsa.paged_workspace_size("norm_rope_bwd", 0, 128), dtype=torch.uint8, device=DEV)
    call = lambda s, ws: dsa.dsa_norm_rope_bwd(s[0], s[1], norm="layer", weight=s[2], with_bias=True, workspace=ws)
    want = [call(s, make()) for s in sets]
    streams, own = [torch.cuda.Stream() for _ in sets], [make() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(call(sets[k], own[k]))
    torch.cuda.synchronize()
    assert all(equal(x, want[k]) for k in range(2) for x in got[k])
    ws = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both = [call(s, ws) for s in sets]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(equal(both[k], want[k]) for k in range(2))
