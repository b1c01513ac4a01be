"""dsa_paged_mla against the 64-bit definition.

Tolerances.  Products of bf16 values are exact in fp32 and sums of 576 of them are off by at most 576 * 2^-24 of the
sum of their magnitudes; with unit-scale inputs and softmax_scale of about 1/24 a score is then off by less than
2^-14, and so is every weight exp(z - lse), relatively; P as bf16 hi + lo leaves 2^-16 of each weight.  An output is
a weighted mean of the values seen: its error is at most 2^-13 of the weighted mean of their magnitudes (bounded here by
the largest one seen), plus half a bf16 step, 2^-8 of itself, for the one rounding.  lse is off by at most the scores'
2^-14 plus a few 2^-24 of its own value."""
import random

import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(lens, news, H, D, page, seed, extra_pages=2, fill=float("nan")):
    """A cache whose unused rows hold `fill`, and requests over randomly placed pages."""
    g = torch.Generator().manual_seed(seed)
    r = random.Random(seed)
    need = [-(-n // page) for n in lens]
    ids = list(range(sum(need) + extra_pages))
    r.shuffle(ids)
    width = max(need + [1]) + 1
    table = [[ids.pop() if c < k else -1 for c in range(width)] for k in need]
    cache = torch.full((sum(need) + extra_pages, page, D), fill, dtype=torch.bfloat16)
    flat = cache.view(-1, D)
    for b, n in enumerate(lens):
        if n:
            flat[ref.rows_of(table[b], range(n), page)] = torch.randn(n, D, generator=g).bfloat16()
    N = sum(news)
    q = torch.randn(N, H, D, generator=g).bfloat16()
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return q, cache, table, cu


def check(got, want, lse, want_lse, most=5.0):
    got, lse = got.cpu().double(), lse.cpu().double()
    inf = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse), inf) and bool((got[inf] == 0).all())
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -13 * most
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / bound).max())
    ok = ~inf
    assert bool(((lse - want_lse)[ok].abs() <= 2.0 ** -14 + 2.0 ** -21 * want_lse[ok].abs()).all())


CASES = [  # lens, new tokens, H, D, page
    ([1], [1], 1, 576, 1),
    ([64], [1], 16, 576, 64),
    ([65], [1], 16, 512, 64),
    ([1000], [1], 64, 576, 16),
    ([5, 1, 130, 64, 63, 129], [1] * 6, 8, 576, 16),
    ([5, 1, 130, 64, 63, 700], [1] * 6, 64, 512, 33),
    ([300, 3, 77], [2, 5, 1], 16, 576, 48),       # a request with fewer positions than new tokens
    ([300, 0, 77, 20], [4, 1, 0, 3], 5, 576, 7),  # an empty request, one without new tokens
    ([300, 400], [4, 3], 24, 576, 64),
    ([300, 400], [2, 3], 40, 512, 128),
    ([500, 200], [2, 1], 128, 576, 64),
    ([500, 200], [1, 1], 100, 576, 64),
    ([3000] * 5, [1] * 5, 64, 576, 64),
    ([700, 90], [70, 90], 16, 576, 64),           # a chunk of a prompt
    ([20] * 700, [1] * 700, 4, 576, 16),          # more requests than CTAs and than threads
    ([20000], [1], 16, 576, 64),
    ([12000, 3], [3, 1], 64, 512, 64),
]


@pytest.mark.parametrize("lens,news,H,D,page", CASES)
@pytest.mark.parametrize("sink", [False, True])
def test_dense(lens, news, H, D, page, sink):
    q, cache, table, cu = make(lens, news, H, D, page, seed=len(lens) + H + D)
    s = torch.randn(H) if sink else None
    scale = D ** -0.5
    want, want_lse = ref.paged_mla(q, cache.nan_to_num(), table, lens, cu, scale, page, s)
    ws = torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV)
    args = (q.to(DEV), cache.to(DEV), dev(table), dev(lens), scale)
    kw = dict(cu_q=dev(cu), attn_sink=None if s is None else s.to(DEV), workspace=ws)
    out, lse = dsa.dsa_paged_mla(*args, **kw)
    check(out, want, lse, want_lse)
    out2, lse2 = dsa.dsa_paged_mla(*args, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    if news == [1] * len(lens):
        out3, lse3 = dsa.dsa_paged_mla(*args, **{**kw, "cu_q": None})
        assert torch.equal(out, out3) and torch.equal(lse, lse3)
    assert dsa.dsa_read_device_status(ws) == 0


@pytest.mark.parametrize("lens,news,H,D,page,K", [([300, 20], [1, 1], 16, 576, 64, 64), ([300, 20, 1], [2, 1, 1], 64, 576, 16, 50),
                                                  ([3000] * 4, [1] * 4, 64, 576, 64, 2048), ([900, 900], [3, 1], 128, 512, 33, 333),
                                                  ([900, 2], [1, 4], 8, 512, 64, 129), ([40] * 500, [1] * 500, 3, 576, 8, 20)])
@pytest.mark.parametrize("with_len", [False, True])
def test_selected(lens, news, H, D, page, K, with_len):
    q, cache, table, cu = make(lens, news, H, D, page, seed=K + H)
    r = random.Random(K)
    rows, cnt = [], []
    for b in range(len(lens)):
        for j in range(news[b]):
            v = ref.visible(lens[b], news[b], j)
            n = min(v, K, r.choice([K, K // 2, 1]))
            pick = r.sample(range(v), n)  # any order
            row = pick + [-1] * (K - n)
            if not with_len:
                r.shuffle(row)  # -1 anywhere
            else:
                row = pick + [0 if v else -1] * (K - n)  # beyond the length: never looked at
            rows.append(row)
            cnt.append(n)
    topk, ln = torch.tensor(rows, dtype=torch.int32), torch.tensor(cnt, dtype=torch.int32)
    sink = torch.randn(H)
    want, want_lse = ref.paged_mla(q, cache.nan_to_num(), table, lens, cu, 0.05, page, sink, topk, ln if with_len else None)
    ws = torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV)
    out, lse = dsa.dsa_paged_mla(q.to(DEV), cache.to(DEV), dev(table), dev(lens), 0.05, cu_q=dev(cu), topk_idx=topk.to(DEV),
                                 topk_len=ln.to(DEV) if with_len else None, attn_sink=sink.to(DEV), workspace=ws)
    check(out, want, lse, want_lse)
    assert dsa.dsa_read_device_status(ws) == 0


def test_a_growing_maximum_rescales():
    # scores that rise along the cache by far more than the threshold, and one token that dominates
    lens, H, D, page = [4000], 64, 576, 64
    q, cache, table, cu = make(lens, [1], H, D, page, seed=4)
    flat = cache.view(-1, D)
    rows = ref.rows_of(table[0], range(4000), page)
    ramp = torch.linspace(0.0, 1.0, 4000)[:, None]
    flat[rows] = (flat[rows].float() * 0.1 + ramp * q[0, 5].float()[None, :]).bfloat16()
    want, want_lse = ref.paged_mla(q, cache.nan_to_num(), table, lens, cu, 0.2, page)
    out, lse = dsa.dsa_paged_mla(q.to(DEV), cache.to(DEV), dev(table), dev(lens), 0.2)
    # (scores up to 0.2 * 576 and more: off by 576 * 2^-24 of the sum of magnitudes, here below 2^-7)
    got = out.cpu().double()
    assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -6 * 0.05).all())
    assert bool(((lse.cpu().double() - want_lse).abs() <= 2.0 ** -7).all())


def test_bad_indices_are_masked_and_reported():
    lens, H, D, page = [200, 100], 16, 576, 16
    q, cache, table, cu = make(lens, [1, 1], H, D, page, seed=6)
    ws = torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV)
    topk = torch.tensor([[3, 200, -2, 7, -1], [99, 100, 2 ** 31 - 1, 0, 5]], dtype=torch.int32)
    want, want_lse = ref.paged_mla(q, cache.nan_to_num(), table, lens, cu, 0.05, page, topk=topk)
    run = lambda **kw: dsa.dsa_paged_mla(q.to(DEV), cache.to(DEV), dev(kw.pop("table", table)), dev(kw.pop("lens", lens)),  # noqa: E731
                                         0.05, workspace=ws, **kw)
    out, lse = run(topk_idx=topk.to(DEV))
    check(out, want, lse, want_lse)
    assert dsa.dsa_read_device_status(ws) == 6
    # a page that does not exist: its positions are masked
    bad = [list(t) for t in table]
    bad[0][2], bad[1][0] = cache.shape[0], -5
    keep0 = [i for i in range(200) if not 32 <= i < 48]
    keep = torch.full((2, 200), -1, dtype=torch.int32)
    keep[0, :len(keep0)] = torch.tensor(keep0, dtype=torch.int32)
    keep[1, :84] = torch.arange(16, 100, dtype=torch.int32)
    want, want_lse = ref.paged_mla(q, cache.nan_to_num(), table, lens, cu, 0.05, page, topk=keep)
    out, lse = run(table=bad)
    check(out, want, lse, want_lse)
    assert dsa.dsa_read_device_status(ws) == 6
    # a length beyond the table: what the table does not hold is masked
    short = [t[:4] for t in table]
    keep = torch.arange(64, dtype=torch.int32)[None].repeat(2, 1)
    want, want_lse = ref.paged_mla(q, cache.nan_to_num(), table, lens, cu, 0.05, page, topk=keep)
    out, lse = run(table=short)
    check(out, want, lse, want_lse)
    assert dsa.dsa_read_device_status(ws) == 6


def test_rows_outside_the_requests_are_left():
    lens, H, D, page = [70, 40], 16, 576, 16
    q, cache, table, cu = make(lens, [2, 1], H, D, page, seed=7)
    q = torch.cat([q, torch.full((5, H, D), float("nan")).bfloat16()])
    out = torch.full((8, H, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((8, H), 4.0, device=DEV)
    for topk in (None, torch.zeros(8, 3, dtype=torch.int32, device=DEV)):
        dsa.dsa_paged_mla(q.to(DEV), cache.to(DEV), dev(table), dev(lens), 0.05, cu_q=dev(cu), out=out, lse=lse, topk_idx=topk)
        assert bool((out[3:] == 3).all()) and bool((lse[3:] == 4).all()) and not bool((lse[:3] == 4).any())


def test_a_nan_stays_in_its_request():
    lens, H, D, page = [700, 640, 650], 64, 576, 64
    q, cache, table, cu = make(lens, [1, 1, 1], H, D, page, seed=8, fill=0.0)
    args = (dev(table), dev(lens), 0.05)
    out, lse = dsa.dsa_paged_mla(q.to(DEV), cache.to(DEV), *args)
    cache.view(-1, D)[ref.rows_of(table[1], [600], page)[0], 3] = float("nan")
    out2, lse2 = dsa.dsa_paged_mla(q.to(DEV), cache.to(DEV), *args)
    assert torch.equal(out[[0, 2]], out2[[0, 2]]) and torch.equal(lse[[0, 2]], lse2[[0, 2]])
    assert bool(out2[1].isnan().all()) and bool(lse2[1].isnan().all())


def test_a_long_cache_past_32_bits_of_bytes():
    # 4.8 GB of cache: row offsets pass 2^31 elements
    D, page, pages = 576, 64, 66000
    cache = torch.empty(pages, page, D, dtype=torch.bfloat16, device=DEV)
    cache.normal_()
    lens = [5000, 300]
    table = torch.stack([torch.arange(pages - 1, pages - 81, -1), torch.arange(40000, 40080)]).to(torch.int32)
    q = torch.randn(2, 16, D).bfloat16()
    rows = [torch.tensor(ref.rows_of(table[b].tolist(), range(lens[b]), page)) for b in range(2)]
    small = torch.cat([cache.view(-1, D)[r.to(DEV)].cpu() for r in rows])
    flat = small.view(-1, 1, D)
    t2 = [list(range(5000)), list(range(5000, 5300)) + [-1] * 4700]
    want, want_lse = ref.paged_mla(q, flat, t2, lens, [0, 1, 2], 0.05, 1)
    out, lse = dsa.dsa_paged_mla(q.to(DEV), cache, table.to(DEV), dev(lens), 0.05)
    check(out, want, lse, want_lse, most=6.0)


def test_a_captured_step_follows_the_lengths():
    H, D, page = 16, 576, 16
    q, cache, table, cu = make([2000, 900], [1, 1], H, D, page, seed=9)
    ws = torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV)
    qd, cd, td, ld = q.to(DEV), cache.to(DEV), dev(table), dev([1, 1])
    dsa.dsa_paged_mla(qd, cd, td, ld, 0.05, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = dsa.dsa_paged_mla(qd, cd, td, ld, 0.05, workspace=ws)
    for lens in ([1, 1], [2000, 900], [64, 65], [0, 700]):
        ld.copy_(dev(lens))
        g.replay()
        want, want_lse = ref.paged_mla(q, cache.nan_to_num(), table, lens, cu, 0.05, page)
        check(out, want, lse, want_lse)
    assert dsa.dsa_read_device_status(ws) == 0


def test_no_tokens():
    e = torch.empty(0, 16, 576, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device=DEV)
    out, lse = dsa.dsa_paged_mla(e, cache, torch.zeros(0, 4, dtype=torch.int32, device=DEV), dev([]), 0.1)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
