"""Attention over a cache of quantised latents against 64 bits: head counts, page sizes, lengths around the tiles' ends,
several new tokens, lists, sinks, rows that see nothing, rows of every scale."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _quant_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def make(bits, D, H, page, lens, news, seed=0, stale=True, spread=0.0, q_scale=1.0, x_scale=1.0):
    """Requests of these lengths (new tokens included) in randomly placed pages; what no request holds is filled with
    0x7f, which no written row has."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    width = ref.layout(D, 512, bits)[3]
    cache = torch.full((pages, page, width), 0x7f if stale else 0, dtype=torch.uint8, device=DEV)
    perm = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(need)) + 1), -9, dtype=I32)
    slots = []
    for b, n in enumerate(lens):
        for c in range(need[b]):
            table[b, c] = perm.pop()
        slots += [int(table[b, p // page]) * page + p % page for p in range(n)]
    x = torch.randn(len(slots), D, generator=g) * x_scale
    if spread:
        x = x * torch.exp2((spread * torch.randn(len(slots), 1, generator=g)).round())
    if slots:
        dsa.dsa_paged_quantize(x.bfloat16().to(DEV), cache, bits, out_rows=torch.tensor(slots, dtype=I32, device=DEV))
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    q = (torch.randn(cu[-1], H, D, generator=g) * q_scale).bfloat16()
    return g, cache, table, q, cu


def run(bits, cache, table, q, lens, cu, scale, topk=None, topk_len=None, sink=None, ws=None, out=None, lse=None):
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    return dsa.dsa_paged_mla_quant(d(q), cache, d(table), torch.tensor(lens, dtype=I32, device=DEV), scale, bits,
                                   cu_q=torch.tensor(cu, dtype=I32, device=DEV), topk_idx=d(topk), topk_len=d(topk_len),
                                   attn_sink=d(sink), out=out, lse=lse, workspace=ws)


def workspace():
    return torch.zeros(dsa.paged_workspace_size("mla_quant"), dtype=torch.uint8, device=DEV)


def compare(bits, D, H, page, lens, news, seed=0, sink=False, scale=None, **kw):
    g, cache, table, q, cu = make(bits, D, H, page, lens, news, seed, **kw)
    s = torch.randn(H, generator=g) if sink else None
    scale = D ** -0.5 if scale is None else scale
    ws = workspace()
    got = run(bits, cache, table, q, lens, cu, scale, sink=s, ws=ws)
    assert dsa.dsa_read_device_status(ws) == 0
    ref.check_attention(got, ref.attention(q, cache, bits, table, lens, cu, scale, s), bits)
    return got


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [576, 512])
@pytest.mark.parametrize("H", [1, 5, 16, 17, 40, 64, 65, 128])
def test_head_counts(bits, D, H):
    compare(bits, D, H, 64, [300, 77], [1, 1], H)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [8, 64])
@pytest.mark.parametrize("lens", [[1], [2, 3], [63, 64, 65], [127, 128, 129], [255, 256, 257], [1000], [0, 5, 0, 400]])
def test_lengths(bits, H, lens):
    compare(bits, 576, H, 16, lens, [1] * len(lens), len(lens), sink=len(lens) == 3)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 100, 128, 1024])
def test_page_sizes(bits, page):
    compare(bits, 576, 24, page, [333, 130], [1, 2], page)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H,lens,news", [(16, [200, 300], [2, 4]), (8, [130, 64], [20, 1]), (64, [260, 3, 90], [3, 5, 0]),
                                         (5, [40, 7, 1, 0], [13, 9, 2, 1]), (128, [150], [4]), (3, [500], [100]),
                                         (32, [129, 131], [2, 3])])
def test_several_new_tokens(bits, H, lens, news):
    """Among them tokens in front of their request's start, which see nothing."""
    compare(bits, 576, H, 32, lens, news, H, sink=H == 8)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H,K,sink", [(64, 300, True), (16, 128, False), (8, 1, False), (40, 129, True), (128, 70, False)])
def test_lists(bits, H, K, sink):
    """In any order, with entries named twice, gaps and lengths; a token with no entry."""
    lens, news = [400, 90, 33], [2, 1, 3]
    g, cache, table, q, cu = make(bits, 576, H, 48, lens, news, K)
    idx = torch.full((6, K), -1, dtype=I32)
    for b in range(3):
        for n in range(cu[b], cu[b + 1]):
            v = lens[b] - news[b] + n - cu[b] + 1
            idx[n] = torch.randint(0, v, (K,), generator=g).to(I32)
    idx[:, 1::5] = -1
    idx[4] = -1
    length = torch.tensor([K, K // 2, K, 0, K, max(1, K - 3)], dtype=I32)
    s = torch.randn(H, generator=g) if sink else None
    ws = workspace()
    got = run(bits, cache, table, q, lens, cu, 0.04, idx, length, s, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    ref.check_attention(got, ref.attention(q, cache, bits, table, lens, cu, 0.04, s, idx, length), bits)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kw", [dict(spread=3.0), dict(spread=12.0, q_scale=0.01), dict(x_scale=2.0 ** 40, q_scale=2.0 ** -40),
                                dict(x_scale=2.0 ** -35, q_scale=2.0 ** 33), dict(q_scale=2.0 ** -60),
                                dict(q_scale=30.0, scale=0.2), dict(x_scale=2.0 ** 45, q_scale=2.0 ** -45, spread=2.0)])
@pytest.mark.parametrize("H", [16, 64])
def test_rows_and_queries_of_every_size(bits, kw, H):
    compare(bits, 576, H, 64, [500, 129], [1, 3], 7, **kw)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [16, 64])
def test_heads_of_very_different_size(bits, H):
    g, cache, table, q, cu = make(bits, 576, H, 64, [300], [2])
    q = (q.float() * torch.exp2(torch.randint(-40, 3, (2, H, 1), generator=g).float())).bfloat16()
    ref.check_attention(run(bits, cache, table, q, [300], cu, 0.1), ref.attention(q, cache, bits, table, [300], cu, 0.1), bits)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [16, 64])
def test_a_maximum_that_rises_late_and_one_that_comes_first(bits, H):
    lens = [700]
    g, cache, table, q, cu = make(bits, 512, H, 64, lens, [1], 3)
    for order in (1, -1):  # scores rise or fall along the request
        x = torch.randn(700, 512, generator=g) + (torch.arange(700)[::1][:, None] * order) * 0.02
        slots = torch.tensor([int(table[0, p // 64]) * 64 + p % 64 for p in range(700)], dtype=I32, device=DEV)
        dsa.dsa_paged_quantize(x.bfloat16().to(DEV), cache, bits, out_rows=slots)
        qq = (q.float().abs() * 0.3).bfloat16()
        ref.check_attention(run(bits, cache, table, qq, lens, cu, 0.05), ref.attention(qq, cache, bits, table, lens, cu, 0.05), bits)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [2, 16, 64])
def test_a_nan_row_reaches_the_tokens_that_see_it(bits, H):
    lens, news = [200], [3]
    g, cache, table, q, cu = make(bits, 576, H, 64, lens, news, 1)
    at = int(table[0, 198 // 64]) * 64 + 198 % 64
    bad = torch.randn(1, 576, generator=g)
    bad[0, 3] = float("nan")
    dsa.dsa_paged_quantize(bad.bfloat16().to(DEV), cache, bits, out_rows=torch.tensor([at], dtype=I32, device=DEV))
    out, lse = run(bits, cache, table, q, lens, cu, 0.04)
    assert bool(torch.isnan(out[1:]).all()) and bool(torch.isnan(lse[1:]).all())
    want = ref.attention(q[:1], cache, bits, table, [198], [0, 1], 0.04)
    ref.check_attention((out[:1], lse[:1]), want, bits)


@pytest.mark.parametrize("bits", [8, 4])
def test_rows_outside_the_requests_are_left(bits):
    g, cache, table, q, cu = make(bits, 576, 16, 16, [30, 40], [2, 1])
    q = torch.randn(8, 16, 576, generator=g).bfloat16()
    out = torch.full((8, 16, 512), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((8, 16), 5.0, device=DEV)
    run(bits, cache, table, q, [30, 40], [2, 4, 5], 0.04, out=out, lse=lse)
    assert bool((out[:2] == 5).all()) and bool((out[5:] == 5).all()) and bool((lse[5:] == 5).all())
    want = ref.attention(q, cache, bits, table, [30, 40], [2, 4, 5], 0.04)
    ref.check_attention((out, lse), want, bits)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("lists", [False, True])
def test_bad_pages_and_positions_are_masked_and_reported(bits, lists):
    lens = [200]
    g, cache, table, q, cu = make(bits, 576, 16, 32, lens, [1])
    idx = torch.arange(200, dtype=I32)[None] if lists else None
    for bad in (-1, cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 2] = bad
        ws = workspace()
        got = run(bits, cache, t, q, lens, cu, 0.04, idx, ws=ws)
        assert dsa.dsa_read_device_status(ws) == 6
        keep = torch.tensor([[p for p in range(200) if p // 32 != 2]], dtype=I32)
        ref.check_attention(got, ref.attention(q, cache, bits, table, lens, cu, 0.04, None, keep), bits)
    if lists:
        idx = torch.tensor([[0, 200, -7, 5, 2 ** 31 - 1, -2 ** 31]], dtype=I32)
        got = run(bits, cache, table, q, lens, cu, 0.04, idx, ws=ws)
        assert dsa.dsa_read_device_status(ws) == 6
        ref.check_attention(got, ref.attention(q, cache, bits, table, lens, cu, 0.04, None, torch.tensor([[0, 5]], dtype=I32)), bits)
    else:  # a request longer than its table
        got = run(bits, cache, table[:, :3].contiguous(), q, lens, cu, 0.04, ws=ws)
        assert dsa.dsa_read_device_status(ws) == 6
        keep = torch.arange(96, dtype=I32)[None]
        ref.check_attention(got, ref.attention(q, cache, bits, table, lens, cu, 0.04, None, keep), bits)


@pytest.mark.parametrize("bits", [8, 4])
def test_many_requests_and_equal_bits(bits):
    lens = [(37 * i) % 410 for i in range(70)]
    news = [1 + i % 3 for i in range(70)]
    g, cache, table, q, cu = make(bits, 576, 16, 16, lens, news, 9)
    first = run(bits, cache, table, q, lens, cu, 0.04)
    ref.check_attention(first, ref.attention(q, cache, bits, table, lens, cu, 0.04), bits)
    ws = workspace()
    for _ in range(3):
        again = run(bits, cache, table, q, lens, cu, 0.04, ws=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("bits,H,n", [(4, 64, 30011), (8, 128, 20000), (4, 8, 70001)])
def test_long_requests(bits, H, n):
    compare(bits, 576, H, 64, [n], [1], 2)


def test_calls_of_nothing():
    ws = workspace()
    q = torch.zeros(0, 16, 576, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(0, 16, 432, dtype=torch.uint8, device=DEV)
    i = torch.zeros(0, dtype=I32, device=DEV)
    out, lse = dsa.dsa_paged_mla_quant(q, cache, i.view(0, 1), i, 0.1, 4, workspace=ws)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
    # requests without anything cached: nothing seen, with and without a sink
    q = torch.ones(2, 16, 576, dtype=torch.bfloat16, device=DEV)
    z = torch.zeros(2, dtype=I32, device=DEV)
    out, lse = dsa.dsa_paged_mla_quant(q, cache, z.view(2, 1), z, 0.1, 4, workspace=ws)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    sink = torch.randn(16, device=DEV)
    out, lse = dsa.dsa_paged_mla_quant(q, cache, z.view(2, 1), z, 0.1, 4, attn_sink=sink, workspace=ws)
    # (through base 2 and back: two roundings of the sink)
    assert bool((out == 0).all()) and bool(((lse - sink).abs() <= 2.0 ** -21 * sink.abs() + 2.0 ** -22).all())
    assert dsa.dsa_read_device_status(ws) == 0
