"""The calls on a quantised cache as a serving loop makes them: captured and replayed while the requests grow, on other
streams, two at a time, with a workspace that graphs share, over caches past 2^32 bytes and requests of the longest length;
rows that were never written, queries that are not finite, waits that run out."""
import math

import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as paged
import _quant_ref as ref
from test_gpu_paged_mla_quant import make, run, workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def dev(v):
    return torch.tensor(v, dtype=I32, device=DEV)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("listed", [False, True])
def test_decode_steps(bits, listed):
    # slots, norm and rotation of the new latents, their quantisation, the attention over them (all, or a list): one graph
    B, H, P, steps = 3, 16, 16, 6
    start, pages, scale = [93, 0, 31], 24, 0.05
    g = torch.Generator().manual_seed(bits)
    width = dsa.paged_quant_row_bytes(576, bits)
    table, order = torch.full((B, 8), -1, dtype=I32), torch.randperm(pages, generator=g).tolist()
    cache, slots = torch.zeros(pages, P, width, dtype=torch.uint8, device=DEV), []
    for b, n in enumerate(start):
        for c in range(-(-n // P)):
            table[b, c] = order.pop()
        slots += paged.rows_of(table[b], range(n), P)
    prompt = torch.randn(len(slots), 576, generator=g).bfloat16().to(DEV)
    dsa.dsa_paged_quantize(prompt, cache, bits, out_rows=dev(slots))
    freq, rscale = dsa.dsa_rope_frequencies(64)
    weight = (1 + 0.1 * torch.randn(512, generator=g)).to(DEV)
    tab, lens, free = table.to(DEV), dev(start), dev(order)
    x = torch.empty(B, 576, dtype=torch.bfloat16, device=DEV)
    q = torch.empty(B, H, 576, dtype=torch.bfloat16, device=DEV)
    idx = torch.full((B, 20), -1, dtype=I32, device=DEV) if listed else None
    small, ws = torch.zeros(256, dtype=torch.uint8, device=DEV), workspace()

    def step():
        at, pos, cu, new_lens, taken = dsa.dsa_paged_slots(lens, tab, free, P, workspace=small)
        lat = dsa.dsa_norm_rope_fwd(x, freq, pos, "rms", 512, weight, rope_scale=rscale, interleaved=True, workspace=small)
        dsa.dsa_paged_quantize(lat, cache, bits, out_rows=at, workspace=small)
        out, lse = dsa.dsa_paged_mla_quant(q, cache, tab, new_lens, scale, bits, topk_idx=idx, workspace=ws)
        return at, lat, new_lens, taken, out, lse

    keep = [t.clone() for t in (cache, tab)]
    x.normal_(), q.normal_()
    step()
    torch.cuda.synchronize()
    for t, s in zip((cache, tab), keep):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        at, lat, new_lens, taken, out, lse = step()
    n = list(start)
    for k in range(steps):
        gg = torch.Generator().manual_seed(100 + k)
        x.copy_(torch.randn(B, 576, generator=gg)), q.copy_(torch.randn(B, H, 576, generator=gg))
        lists = torch.full((B, 20), -1, dtype=I32)
        for b in range(B):
            n[b] += 1
            some = torch.randperm(n[b], generator=gg)[:19].tolist()
            lists[b, :len(some)] = torch.tensor(some, dtype=I32)
        if listed:
            idx.copy_(lists)
        before = cache.clone()
        graph.replay()
        assert new_lens.tolist() == n
        rows = at.tolist()
        assert torch.equal(cache.view(-1, width)[rows].cpu(), ref.encode(lat.cpu(), 512, bits))
        other = torch.ones(pages * P, dtype=torch.bool)
        other[rows] = False
        assert torch.equal(cache.view(-1, width)[other.to(DEV)], before.view(-1, width)[other.to(DEV)])
        want = ref.attention(q.cpu(), cache, bits, tab.cpu(), n, list(range(B + 1)), scale, topk=lists if listed else None)
        ref.check_attention((out, lse), want, bits)
        lens.copy_(new_lens)
        free.copy_(torch.roll(free, -int(taken)))
    assert dsa.dsa_read_device_status(ws) == 0 and dsa.dsa_read_device_status(small) == 0


def case(bits, seed, H=64, lens=(900, 863, 64, 700)):
    g, cache, table, q, cu = make(bits, 576, H, 16, list(lens), [1] * len(lens), seed)
    return dict(cache=cache, table=table.to(DEV), q=q.to(DEV), lens=dev(list(lens)), bits=bits)


def attend(s, ws, **kw):
    return dsa.dsa_paged_mla_quant(s["q"], s["cache"], s["table"], s["lens"], 0.04, s["bits"], workspace=ws, **kw)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [8, 4])
def test_two_calls_at_once(bits):
    sets = [case(bits, 1), case(bits, 2, 16)]
    want = [attend(s, workspace()) for s in sets]
    own = [workspace() for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(attend(sets[k], own[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(same(x, want[k]) for x in got[k])
        assert dsa.dsa_read_device_status(own[k]) == 0


def test_graphs_that_share_a_workspace():
    # graphs of both widths, and of the bf16 call, whose workspace is as large
    sets = [case(8, 3), case(4, 4), case(4, 5, 16)]
    bf = dict(q=sets[0]["q"], cache=torch.randn(*sets[0]["cache"].shape[:2], 576, device=DEV).bfloat16())
    ws = torch.zeros(max(dsa.paged_workspace_size("mla"), dsa.paged_workspace_size("mla_quant")), dtype=torch.uint8, device=DEV)

    def call(k, w):
        if k < 3:
            return attend(sets[k], w)
        return dsa.dsa_paged_mla(bf["q"], bf["cache"], sets[0]["table"], sets[0]["lens"], 0.04, workspace=w)
    want = [call(k, torch.zeros_like(ws)) for k in range(4)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for k in range(4):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call(k, ws))
        graphs.append(g)
    for k in (0, 1, 2, 3, 3, 2, 1, 0, 2, 0):
        for t in got[k]:
            t.zero_()
        graphs[k].replay()
        assert same(got[k], want[k])
    assert dsa.dsa_read_device_status(ws) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_a_captured_call_follows_the_lengths(bits):
    s = case(bits, 6, 40, (2000, 900))
    lens, ws = s["lens"], workspace()
    attend(s, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = attend(s, ws)
    for now in ([1, 1], [2000, 900], [96, 97], [64, 65], [0, 700]):
        lens.copy_(dev(now))
        g.replay()
        want = ref.attention(s["q"].cpu(), s["cache"], bits, s["table"].cpu(), now, [0, 1, 2], 0.04)
        ref.check_attention(got, want, bits)
    assert dsa.dsa_read_device_status(ws) == 0


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [16, 64])
def test_rows_that_were_never_written_hold_zeros(bits, H):
    # pages of zero bytes: every score 0, the output 0, the weights even; and beside written rows
    lens = [150, 200]
    g, cache, table, q, cu = make(bits, 576, H, 16, lens, [1, 1], 7)
    flat = cache.view(-1, cache.shape[2])
    for b, n in ((0, 150), (1, 77)):
        flat[torch.tensor(paged.rows_of(table[b].tolist(), range(n), 16), device=DEV)] = 0
    got = run(bits, cache, table, q, lens, cu, 0.04)
    ref.check_attention(got, ref.attention(q, cache, bits, table, lens, cu, 0.04), bits)
    # (the least s goes into the sum's logarithm and out of it again: numbers of up to 53 ln 2, a few roundings)
    assert bool((got[0][0] == 0).all()) and bool(((got[1][0] - math.log(150)).abs() <= 2.0 ** -16).all())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [4, 16, 64])
def test_a_query_that_is_not_finite_stays_in_its_row(bits, H):
    lens, news = [200, 70], [4, 2]
    g, cache, table, q, cu = make(bits, 576, H, 64, lens, news, H)
    want = ref.attention(q, cache, bits, table, lens, cu, 0.04)
    q[0], q[4, 0], q[5, H - 1, 3], q[2, 1, 575] = float("nan"), float("inf"), -float("inf"), float("nan")
    bad = torch.zeros(6, H, dtype=torch.bool)
    bad[0], bad[4, 0], bad[5, H - 1], bad[2, 1] = True, True, True, True
    out, lse = run(bits, cache, table, q, lens, cu, 0.04)
    nan = torch.zeros(6, H, dtype=torch.bool)
    nan[0], nan[2, 1] = True, True
    assert bool(out.cpu()[nan].isnan().all()) and bool(lse.cpu()[nan].isnan().all())
    assert not bool(torch.isfinite(lse.cpu()[bad]).any())
    want[1][bad] = float("nan")
    ref.check_attention((out, lse), want, bits)


def test_a_position_named_twice_counts_twice():
    for bits in (8, 4):
        s = case(bits, 8, 16, (40,))
        got = attend(s, workspace(), topk_idx=dev([[5, 5, 9]]))
        want = ref.attention(s["q"].cpu(), s["cache"], bits, s["table"].cpu(), [40], [0, 1], 0.04,
                             topk=torch.tensor([[5, 5, 9]]))
        ref.check_attention(got, want, bits)


@pytest.mark.parametrize("bits", [8, 4])
def test_a_cache_past_32_bits_of_bytes(bits):
    # two requests' rows at both ends of a cache of more than 2^32 bytes; written, attended and read back
    page, width = 64, dsa.paged_quant_row_bytes(576, bits)
    pages = 2 ** 32 // (page * width) + 200
    cache = torch.empty(pages, page, width, dtype=torch.uint8, device=DEV)
    lens = [3000, 300]
    table = torch.stack([torch.arange(pages - 1, pages - 81, -1), torch.arange(7, 87)]).to(I32)
    rows = [paged.rows_of(table[b].tolist(), range(lens[b]), page) for b in range(2)]
    assert max(rows[0]) * width > 2 ** 32
    g = torch.Generator().manual_seed(3)
    x = torch.randn(sum(lens), 576, generator=g).bfloat16()
    dsa.dsa_paged_quantize(x.to(DEV), cache, bits, out_rows=dev(rows[0] + rows[1]))
    small = torch.zeros(sum(lens), 1, width, dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(x.to(DEV), small, bits, out_rows=dev(list(range(sum(lens)))))
    cu = dev([0, 3000, 3300])
    back = dsa.dsa_paged_dequantize(cache, table.to(DEV), cu, bits, 576, N=3300)
    assert torch.equal(back, dsa.dsa_paged_dequantize(small, torch.arange(3300, dtype=I32, device=DEV)[None],
                                                      dev([0, 3300]), bits, 576, N=3300))
    q = torch.randn(2, 16, 576, generator=g).bfloat16()
    t2 = torch.full((2, 3000), -1, dtype=I32)
    t2[0], t2[1, :300] = torch.arange(3000, dtype=I32), torch.arange(3000, 3300, dtype=I32)
    for k in (None, torch.arange(0, 300, 7, dtype=I32).repeat(2, 1)):
        got = run(bits, cache, table, q, lens, [0, 1, 2], 0.04, topk=k)
        ref.check_attention(got, ref.attention(q, small, bits, t2, lens, [0, 1, 2], 0.04, topk=k), bits)
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bits", [8, 4])
def test_a_request_of_the_longest_length(bits):
    # 2^31 - 1 positions in one page of 64 that the table names again and again; every CTA adds its 2^25 / 152 tiles of 64
    # (or fewer of 96) one after the other: sums of positive terms, each addition off by at most 2^-24 of the sum
    g = torch.Generator().manual_seed(5)
    cache = torch.zeros(1, 64, dsa.paged_quant_row_bytes(512, bits), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(torch.randn(64, 512, generator=g).bfloat16().to(DEV), cache, bits)
    q = torch.randn(1, 1, 512, generator=g).bfloat16()
    ws = workspace()
    out, lse = dsa.dsa_paged_mla_quant(q.to(DEV), cache, torch.zeros(1, 2 ** 25, dtype=I32, device=DEV), dev([2 ** 31 - 1]),
                                       0.04, bits, workspace=ws)
    _, one, *_ = ref.attention(q, cache, bits, torch.zeros(1, 1, dtype=I32), [64], [0, 1], 0.04)
    # (one position of 2^31 is missing, which is nothing beside the sums' errors)
    assert abs(float(lse) - (25 * math.log(2) + float(one))) <= 2 ** 25 / 152 * 2.0 ** -24 + 2.0 ** -12
    assert bool(torch.isfinite(out).all()) and dsa.dsa_read_device_status(ws) == 0


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("lists", [False, True])
def test_thousands_of_short_requests(bits, lists):
    B, H, page, pool = 1600, 3, 8, 400
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(0, 110, (B,), generator=g)
    table = torch.full((B, 14), -1, dtype=I32)
    for b in range(B):
        k = -(-int(lens[b]) // page)
        table[b, :k] = torch.randint(0, pool, (k,), generator=g, dtype=I32)
    cache = torch.zeros(pool, page, dsa.paged_quant_row_bytes(576, bits), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(torch.randn(pool * page, 576, generator=g).bfloat16().to(DEV), cache, bits,
                           out_rows=torch.arange(pool * page, dtype=I32, device=DEV))
    q = torch.randn(B, H, 576, generator=g).bfloat16()
    idx = None
    if lists:
        idx = (torch.rand(B, 6, generator=g) * lens.clamp(min=1)[:, None]).to(I32)
        idx[lens == 0] = -1
    ws = workspace()
    got = run(bits, cache, table, q, lens.tolist(), list(range(B + 1)), 0.04, topk=idx, ws=ws)
    ref.check_attention(got, ref.attention(q, cache, bits, table, lens.tolist(), list(range(B + 1)), 0.04, topk=idx), bits)
    assert dsa.dsa_read_device_status(ws) == 0


@pytest.fixture
def zero_wait_limit():
    dsa.dsa_set_wait_limit_cycles(0)
    try:
        yield
    finally:
        dsa.dsa_set_wait_limit_cycles(-1)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H,page,listed", [(64, 64, False), (16, 16, False), (64, 13, False), (64, 64, True)])
def test_waits_of_no_time(zero_wait_limit, bits, H, page, listed):
    # every CTA gives up at its first wait, leaves cleanly and reports it; the next call gives the right answer again
    lens = [3000, 700, 64]
    g, cache, table, q, cu = make(bits, 576, H, page, lens, [1, 1, 1], H)
    topk = torch.tensor([[(7 * i) % n for i in range(50)] for n in lens], dtype=I32) if listed else None
    ws = workspace()
    for _ in range(3):
        run(bits, cache, table, q, lens, cu, 0.05, topk=topk, ws=ws)
        assert dsa.dsa_read_device_status(ws) == 7
    dsa.dsa_set_wait_limit_cycles(-1)
    got = run(bits, cache, table, q, lens, cu, 0.05, topk=topk, ws=ws)
    ref.check_attention(got, ref.attention(q, cache, bits, table, lens, cu, 0.05, topk=topk), bits)
    assert dsa.dsa_read_device_status(ws) == 0


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("limit", [100, 1000, 2000, 4000, 8000, 16000, 40000])
def test_waits_that_run_out_somewhere(zero_wait_limit, bits, limit):
    # the roles give up at different places, some CTAs not at all; every call ends and says whether its results count
    lens = [3000, 700, 64, 1500, 20]
    g, cache, table, q, cu = make(bits, 576, 64, 64, lens, [1] * 5, limit)
    topk = torch.tensor([[(11 * i) % n for i in range(300)] for n in lens], dtype=I32)
    ws = workspace()
    for k in (None, topk):
        dsa.dsa_set_wait_limit_cycles(-1)
        want = run(bits, cache, table, q, lens, cu, 0.05, topk=k, ws=ws)
        torch.cuda.synchronize()
        dsa.dsa_set_wait_limit_cycles(limit)
        for _ in range(8):
            got = run(bits, cache, table, q, lens, cu, 0.05, topk=k, ws=ws)
            status = dsa.dsa_read_device_status(ws)
            assert status in (0, 7) and (status == 7 or same(got, want))
