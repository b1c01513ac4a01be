"""The bounded waits of the paged attention and selection: with a limit of 0 cycles every CTA gives up at its first wait,
leaves cleanly and reports DSA_ERR_TIMEOUT (its results are not defined and not looked at); the next call with the default
limit gives the right answer again."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref
from test_gpu_paged_indexer import make as make_keys
from test_gpu_paged_mla import check, dev, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture
def zero_wait_limit():
    dsa.dsa_set_wait_limit_cycles(0)
    try:
        yield
    finally:
        dsa.dsa_set_wait_limit_cycles(-1)


@pytest.mark.parametrize("H,page,listed", [(64, 64, False), (16, 16, False), (64, 33, False), (64, 64, True)])
def test_attention(zero_wait_limit, H, page, listed):
    lens = [3000, 700, 64]
    q, cache, table, cu = make(lens, [1, 1, 1], H, 576, page, seed=H)
    topk = torch.tensor([[(7 * i) % n for i in range(50)] for n in lens], dtype=torch.int32) if listed else None
    ws = torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV)
    args = (q.to(DEV), cache.to(DEV), dev(table), dev(lens), 0.05)
    kw = dict(topk_idx=None if topk is None else topk.to(DEV), workspace=ws)
    for _ in range(3):
        dsa.dsa_paged_mla(*args, **kw)
        assert dsa.dsa_read_device_status(ws) == 7
    dsa.dsa_set_wait_limit_cycles(-1)
    want, want_lse = ref.paged_mla(q, cache.nan_to_num(), table, lens, cu, 0.05, page, topk=topk)
    out, lse = dsa.dsa_paged_mla(*args, **kw)
    check(out, want, lse, want_lse)
    assert dsa.dsa_read_device_status(ws) == 0


@pytest.mark.parametrize("page", [64, 33])
def test_selection(zero_wait_limit, page):
    lens, K = [3000, 700, 64], 50
    q, k, w, table, cu = make_keys(lens, [1, 1, 1], 64, page, seed=1)
    ws = torch.zeros(dsa.paged_workspace_size("topk", 3, len(table[0]) * page), dtype=torch.uint8, device=DEV)
    args = (q.to(DEV), k.to(DEV), w.to(DEV), dev(table), dev(lens), K)
    for _ in range(3):
        dsa.dsa_paged_indexer_topk(*args, workspace=ws)
        assert dsa.dsa_read_device_status(ws) == 7
    dsa.dsa_set_wait_limit_cycles(-1)
    idx, ln = dsa.dsa_paged_indexer_topk(*args, workspace=ws)
    assert dsa.dsa_read_device_status(ws) == 0
    for b in range(3):
        want = ref.topk_of(ref.paged_scores(q[b], k, w[b], table[b], lens[b], page)[0], K)
        assert idx[b].tolist() == want + [-1] * (K - len(want))


@pytest.mark.parametrize("limit", [100, 400, 1000, 2000, 4000, 8000, 16000, 40000])
def test_waits_that_run_out_somewhere(zero_wait_limit, limit):
    # a limit of some tiles' time: the roles give up at different places, some CTAs not at all; every call ends and says
    # whether its results count
    lens = [3000, 700, 64, 1500, 20]
    q, cache, table, cu = make(lens, [1] * 5, 64, 576, 64, seed=limit)
    topk = torch.tensor([[(11 * i) % n for i in range(300)] for n in lens], dtype=torch.int32)
    qi, k, w, ktable, _ = make_keys(lens, [1] * 5, 64, 64, seed=limit)
    ws = torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV)
    wt = torch.zeros(dsa.paged_workspace_size("topk", 5, len(ktable[0]) * 64), dtype=torch.uint8, device=DEV)
    args = (q.to(DEV), cache.to(DEV), dev(table), dev(lens), 0.05)
    targs = (qi.to(DEV), k.to(DEV), w.to(DEV), dev(ktable), dev(lens), 50)
    dense, listed = dict(workspace=ws), dict(workspace=ws, topk_idx=topk.to(DEV))
    want = [dsa_default(lambda: dsa.dsa_paged_mla(*args, **kw), limit) for kw in (dense, listed)]
    lists = dsa_default(lambda: dsa.dsa_paged_indexer_topk(*targs, workspace=wt), limit)
    for _ in range(8):
        for kw, right in zip((dense, listed), want):
            out, lse = dsa.dsa_paged_mla(*args, **kw)
            status = dsa.dsa_read_device_status(ws)
            assert status in (0, 7)
            if status == 0:
                assert torch.equal(out, right[0]) and torch.equal(lse, right[1])
        idx, n = dsa.dsa_paged_indexer_topk(*targs, workspace=wt)
        status = dsa.dsa_read_device_status(wt)
        assert status in (0, 7) and (status == 7 or torch.equal(idx, lists[0]))


def dsa_default(call, limit):
    """The call with the default limit; then the limit is `limit`."""
    dsa.dsa_set_wait_limit_cycles(-1)
    got = call()
    torch.cuda.synchronize()
    dsa.dsa_set_wait_limit_cycles(limit)
    return got
