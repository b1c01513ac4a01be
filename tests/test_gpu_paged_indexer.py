"""dsa_paged_indexer_topk against the definition in 64 bits.

On a grid of values whose every sum is exact in fp32 (multiples of 1/8 up to 3 and weights that are multiples of 1/1024:
products are multiples of 2^-16, sums stay below 2^7) the lists have to be equal, ties included.  On unit-scale values the
sets may differ only where |score - K-th score| is within 200 * 2^-24 of the two sums of magnitudes (128 products, 64
heads: fewer than 200 additions)."""
import random

import numpy as np
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(lens, news, Hi, page, seed, grid=True):
    g = torch.Generator().manual_seed(seed)
    r = random.Random(seed)
    need = [-(-n // page) for n in lens]
    ids = list(range(sum(need) + 3))
    r.shuffle(ids)
    width = max(need + [1]) + 1
    table = [[ids.pop() if c < k else -1 for c in range(width)] for k in need]
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    q, k = torch.randn(cu[-1], Hi, 128, generator=g), torch.randn(sum(need) + 3, page, 128, generator=g)
    w = torch.rand(cu[-1], Hi, generator=g) - 0.25
    if grid:
        q, k = [((x * 8).round() / 8).clamp(-3, 3) for x in (q, k)]
        w = (w * 128).round() / 1024
    return q.bfloat16(), k.bfloat16(), w, table, cu


def run(q, k, w, table, lens, cu, K, **kw):
    ws = torch.zeros(dsa.paged_workspace_size("topk", q.shape[0], len(table[0]) * k.shape[1]), dtype=torch.uint8, device=DEV)
    idx, ln = dsa.dsa_paged_indexer_topk(q.to(DEV), k.to(DEV), w.to(DEV), dev(table), dev(lens), K,
                                         cu_q=None if cu is None else dev(cu), workspace=ws, **kw)
    assert dsa.dsa_read_device_status(ws) == 0
    return idx.cpu().numpy(), ln.cpu().numpy()


CASES = [  # lens, new tokens, heads, page, K
    ([1], [1], 64, 64, 1),
    ([1], [1], 1, 1, 2048),
    ([129], [1], 64, 16, 128),
    ([130, 1, 300], [1, 1, 1], 64, 64, 64),
    ([130, 2, 300, 0], [2, 4, 3, 1], 32, 48, 50),   # fewer positions than new tokens; an empty request
    ([600, 40, 7], [9, 0, 7], 5, 33, 77),
    ([5000, 2049, 2048], [1, 2, 1], 64, 64, 2048),
    ([300] * 400, [1] * 400, 16, 64, 17),
    ([900, 200], [300, 200], 8, 16, 100),           # a chunk of a prompt
]


@pytest.mark.parametrize("lens,news,Hi,page,K", CASES)
def test_lists_on_a_grid_are_equal(lens, news, Hi, page, K):
    q, k, w, table, cu = make(lens, news, Hi, page, seed=K + Hi)
    idx, ln = run(q, k, w, table, lens, cu, K)
    for b in range(len(lens)):
        for n in range(cu[b], cu[b + 1]):
            v = ref.visible(lens[b], news[b], n - cu[b])
            want = ref.topk_of(ref.paged_scores(q[n], k, w[n], table[b], v, page)[0], K) if v else []
            assert ln[n] == len(want) and idx[n].tolist() == want + [-1] * (K - len(want)), (b, n)
    idx2, ln2 = run(q, k, w, table, lens, cu, K)
    assert np.array_equal(idx, idx2) and np.array_equal(ln, ln2)


# lengths on both sides of what one, two, four and eight CTAs hold, and beyond what they hold in one round
@pytest.mark.parametrize("L,K", [(4097, 2048), (8200, 100), (16384, 2048), (16389, 2048), (40000, 1), (70001, 2048),
                                 (131072, 2048), (131077, 2047), (300001, 2048)])
@pytest.mark.parametrize("ties", [False, True])
def test_long_rows(L, K, ties):
    q, k, w, table, cu = make([L], [1], 8, 64, seed=L, grid=True)
    if ties:  # few distinct scores: whole runs of equal ones
        k = k * 0
        k[..., 0] = (torch.randint(0, 3, k.shape[:2], generator=torch.Generator().manual_seed(L))).bfloat16()
        q, w = torch.ones_like(q), torch.ones_like(w)
    idx, ln = run(q, k, w, table, [L], None, K)
    rows = k.double().reshape(-1, 128)[ref.rows_of(table[0], range(L), 64)]
    s = (w[0].double()[:, None] * (q[0].double() @ rows.T).clamp(min=0)).sum(0).numpy()
    want = np.sort(np.argsort(-s, kind="stable")[:K])
    assert ln[0] == K and np.array_equal(idx[0], want)


def test_unit_scale_sets_up_to_the_tie_band():
    lens, news, K = [3000, 900, 5000], [2, 1, 1], 256
    q, k, w, table, cu = make(lens, news, 64, 64, seed=3, grid=False)
    idx, ln = run(q, k, w, table, lens, cu, K)
    for b in range(3):
        for n in range(cu[b], cu[b + 1]):
            v = ref.visible(lens[b], news[b], n - cu[b])
            s, mag = ref.paged_scores(q[n], k, w[n], table[b], v, 64)
            want = ref.topk_of(s, K)
            got = idx[n, :ln[n]].tolist()
            assert len(got) == len(want) and got == sorted(set(got))
            kth = min(want, key=lambda i: float(s[i]))
            for d in set(got) ^ set(want):
                assert abs(float(s[d] - s[kth])) <= 200 * 2.0 ** -24 * float(mag[d] + mag[kth])


def test_values_that_are_not_finite():
    # NaN ranks above all, then +inf; negative scores are ranked like others
    q, k, w, table, cu = make([500], [1], 4, 64, seed=5)
    rows = ref.rows_of(table[0], range(500), 64)
    flat = k.view(-1, 128)
    q[:] = 1.0
    w[:] = -1.0
    w[0, 0] = 1.0
    flat[rows[17], 0] = float("nan")
    flat[rows[400], 0] = float("nan")
    idx, ln = run(q, k, w, table, [500], cu, 2)
    assert idx[0].tolist() == [17, 400]
    s, _ = ref.paged_scores(q[0], k.nan_to_num(), w[0], table[0], 500, 64)
    s[[17, 400]] = float("inf")
    idx, ln = run(q, k, w, table, [500], cu, 100)
    assert idx[0].tolist() == ref.topk_of(s, 100)


def test_bad_pages_short_bounds_and_rows_that_are_left():
    lens, page, K = [300, 90], 64, 60
    q, k, w, table, cu = make(lens, [1, 1], 64, page, seed=9)
    ws = torch.zeros(dsa.paged_workspace_size("topk", 4, 512), dtype=torch.uint8, device=DEV)
    w = w.abs()

    def go(table, lens, **kw):
        idx, ln = dsa.dsa_paged_indexer_topk(q.to(DEV), k.to(DEV), w.to(DEV), dev(table), dev(lens), K, workspace=ws, **kw)
        return idx.tolist(), ln.tolist()

    bad = [list(t) for t in table]
    bad[0][1] = k.shape[0]
    idx, ln = go(bad, lens)
    s, _ = ref.paged_scores(q[0], k, w[0], [t if i != 1 else 0 for i, t in enumerate(table[0])], 300, page)
    s[64:128] = 0.0  # rows of zeros
    assert idx[0] == ref.topk_of(s, K) and dsa.dsa_read_device_status(ws) == 6
    idx, ln = go(table, lens, max_len=100)
    s, _ = ref.paged_scores(q[0], k, w[0], table[0], 100, page)
    assert idx[0] == ref.topk_of(s, K) and dsa.dsa_read_device_status(ws) == 6
    # tokens after the last request
    q4, w4 = torch.cat([q, q]), torch.cat([w, w])
    out, ol = torch.full((4, K), 9, dtype=torch.int32, device=DEV), torch.full((4,), 9, dtype=torch.int32, device=DEV)
    dsa.dsa_paged_indexer_topk(q4.to(DEV), k.to(DEV), w4.to(DEV), dev(table), dev(lens), K, cu_q=dev([0, 1, 2]),
                               topk_idx=out, topk_len=ol, workspace=ws)
    assert bool((out[2:] == 9).all()) and ol.tolist() == [60, 60, 9, 9] and not bool((out[:2] == 9).all())
    assert dsa.dsa_read_device_status(ws) == 0


def test_a_captured_selection_follows_the_lengths():
    q, k, w, table, cu = make([40000, 900], [1, 1], 64, 64, seed=12)
    a = (q.to(DEV), k.to(DEV), w.to(DEV), dev(table))
    ld = dev([1, 1])
    ws = torch.zeros(dsa.paged_workspace_size("topk", 2, len(table[0]) * 64), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_indexer_topk(*a, ld, 512, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx, ln = dsa.dsa_paged_indexer_topk(*a, ld, 512, workspace=ws)
    for lens in ([40000, 900], [3, 513], [5000, 0]):
        ld.copy_(dev(lens))
        g.replay()
        for b in range(2):
            s = ref.paged_scores(q[b], k, w[b], table[b], lens[b], 64)[0] if lens[b] else []
            want = ref.topk_of(s, 512)
            assert ln[b].item() == len(want) and idx[b].tolist() == want + [-1] * (512 - len(want))
    assert dsa.dsa_read_device_status(ws) == 0


def test_no_tokens():
    e = torch.empty(0, 64, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(2, 16, 128, dtype=torch.bfloat16, device=DEV)
    idx, ln = dsa.dsa_paged_indexer_topk(e, k, torch.empty(0, 64, device=DEV), torch.zeros(0, 4, dtype=torch.int32, device=DEV),
                                         dev([]), 16)
    assert idx.shape == (0, 16) and ln.shape == (0,)
