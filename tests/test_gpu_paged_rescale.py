"""dsa_paged_mla where the running maximum rises inside a CTA's run of tiles, in its last tile too, so that the sums and
the outputs formed before are scaled.

A request's scores lie near 0 but for some positions that lie about 7 higher (10 in log2, past the threshold of a raise, 8):
one at its end, or one in every tile, each 7 above the one before.  120 requests of 10 tiles and more lie on every CTA's
range about one by one, so a run has several tiles, wherever it is cut.

Tolerances.  A score is a sum of D products, exact in fp32: off by at most D 2^-24 of the sum of their magnitudes, which
is formed below (`mag`); a weight is off by twice that, relatively (its own score and the sum's), and by 2^-16 as bf16
hi + lo; sums of 700 positive terms in fp32 by 700 2^-24 < 2^-14.  An output is off by that share of the largest value of
its channel, plus half a bf16 step for its rounding; lse by the score's error and 2^-14, and 2^-22 of itself."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B = 120


def dev(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(H, D, page, every, seed):
    g = torch.Generator().manual_seed(seed)
    lens = [640 + b % 60 for b in range(B)]
    width = -(-700 // page)
    table = torch.randperm(B * width, generator=g).view(B, width)
    q = 0.25 * torch.randn(B, H, D, generator=g)
    q[..., D - 1] = 8.0 + torch.randint(0, 4, (B, H), generator=g) / 4
    cache = 0.5 * torch.randn(B * width, page, D, generator=g)
    cache[..., D - 1] = 0.0
    flat = cache.view(-1, D)
    for b, n in enumerate(lens):
        top = range(63, n, 64) if every else [n - 1]
        for k, p in enumerate(top):
            flat[ref.rows_of(table[b], [p], page)[0], D - 1] = 17.0 * (k + 1)
    return q.bfloat16(), cache.bfloat16(), table.tolist(), lens


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("D,page,lists", [(576, 64, False), (512, 64, False), (576, 33, False), (576, 64, True), (512, 16, True)])
@pytest.mark.parametrize("every", [False, True])
def test_a_maximum_that_rises_in_a_run(H, D, page, lists, every):
    q, cache, table, lens = make(H, D, page, every, seed=H + D + page)
    scale = 0.05
    topk = None
    if lists:  # every position, the raising ones where they are in the dense form
        topk = torch.full((B, 700), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            topk[b, :n] = torch.arange(n, dtype=torch.int32)
    want, want_lse = ref.paged_mla(q, cache, table, lens, list(range(B + 1)), scale, page, None, topk)
    rows = [ref.rows_of(table[b], range(n), page) for b, n in enumerate(lens)]
    mag = torch.stack([(q[b].double().abs() @ cache.view(-1, D)[rows[b]].double().abs().T).amax(1) for b in range(B)]) * scale
    off = D * 2.0 ** -24 * mag[..., None]
    big = torch.stack([cache.view(-1, D)[rows[b], :512].double().abs().amax(0) for b in range(B)])[:, None, :]
    ws = torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV)
    args = (q.to(DEV), cache.to(DEV), dev(table), dev(lens), scale)
    kw = dict(topk_idx=None if topk is None else topk.to(DEV), workspace=ws)
    out, lse = dsa.dsa_paged_mla(*args, **kw)
    got, got_lse = out.cpu().double(), lse.cpu().double()
    bound = 2.0 ** -8 * want.abs() + (2 * off + 2.0 ** -14) * big
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / bound).max())
    assert bool(((got_lse - want_lse).abs() <= off[..., 0] + 2.0 ** -14 + 2.0 ** -22 * want_lse.abs()).all())
    for _ in range(20):  # whatever the order in which the warps came
        again, lse2 = dsa.dsa_paged_mla(*args, **kw)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert dsa.dsa_read_device_status(ws) == 0
