"""dsa_paged_mla over latents that are not finite, at positions that some of a request's new tokens see and others do not: the
tokens that do not see them get what they get without them, by the definition in 64 bits (tolerances as in test_gpu_paged_mla.py,
whose helpers are used: unit-scale values); the ones that see them do not hide them."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref
from test_gpu_paged_mla import check, dev, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")

CASES = [  # lens, new tokens, H, D, page
    ([130, 65, 300], [2, 3, 4], 1, 576, 64),
    ([130, 65, 300], [2, 3, 4], 8, 512, 64),
    ([130, 64, 700], [2, 4, 4], 16, 576, 16),
    ([130, 64, 700], [2, 3, 2], 24, 576, 64),
    ([129, 9000, 66], [2, 2, 3], 64, 576, 64),
    ([129, 500, 66], [2, 2, 3], 100, 512, 33),
    ([129, 500, 66], [2, 4, 3], 128, 576, 64),
    ([200, 100], [70, 100], 1, 576, 64),      # chunks of prompts, many tokens a group
    ([200, 100], [70, 100], 8, 512, 33),
]


def run(q, cache, table, lens, cu, D):
    ws = torch.zeros(dsa.paged_workspace_size("mla"), dtype=torch.uint8, device=DEV)
    out, lse = dsa.dsa_paged_mla(q.to(DEV), cache.to(DEV), dev(table), dev(lens), D ** -0.5, cu_q=dev(cu), workspace=ws)
    assert dsa.dsa_read_device_status(ws) == 0
    return out.cpu(), lse.cpu()


@pytest.mark.parametrize("lens,news,H,D,page", CASES)
@pytest.mark.parametrize("value", [float("nan"), INF, -INF])
@pytest.mark.parametrize("channel", [3, -1])  # of the values, and past them where the width is 576
def test_a_latent_reaches_the_tokens_that_see_it(lens, news, H, D, page, value, channel):
    q, cache, table, cu = make(lens, news, H, D, page, seed=H + D, fill=0.0)
    want, want_lse = ref.paged_mla(q, cache, table, lens, cu, D ** -0.5, page)
    bad = cache.clone()
    free = []  # the tokens that do not see the bad position
    for b, n in enumerate(lens):
        at = n - 1 - (news[b] - 1) // 2
        bad.view(-1, D)[ref.rows_of(table[b], [at], page)[0], channel] = value
        free += [cu[b] + j for j in range(news[b]) if ref.visible(n, news[b], j) <= at]
    out, lse = run(q, bad, table, lens, cu, D)
    assert free
    check(out[free], want[free], lse[free], want_lse[free])
    seen = [t for t in range(cu[-1]) if t not in free]
    if value != value:
        assert bool(out[seen].isnan().all()) and bool(lse[seen].isnan().all())
        return
    # a score of +inf: NaN; of -inf: what the other positions give (or NaN in the channel of the infinite value)
    up = (q[seen][..., channel].float() * value > 0)
    assert bool(out[seen][up].isnan().all()) and not bool(lse[seen][up].isfinite().any())
    down = (q[seen][..., channel].float() * value < 0)
    listed = torch.full((cu[-1], max(lens)), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        at = n - 1 - (news[b] - 1) // 2
        keep = torch.tensor([p for p in range(n) if p != at], dtype=torch.int32)
        for j in range(news[b]):
            mine = keep[keep < ref.visible(n, news[b], j)]
            listed[cu[b] + j, :len(mine)] = mine
    less, less_lse = ref.paged_mla(q, cache, table, lens, cu, D ** -0.5, page, topk=listed)
    got = out[seen].double()
    at = channel % D
    if at < 512:
        got[..., at] = torch.where(got[..., at].isnan(), less[seen][..., at], got[..., at])
    check(got[down], less[seen][down], lse[seen][down], less_lse[seen][down])


@pytest.mark.parametrize("H", [4, 16, 64])
def test_a_query_that_is_not_finite_stays_in_its_row(H):
    lens, news, D, page = [200, 70], [4, 2], 576, 64
    q, cache, table, cu = make(lens, news, H, D, page, seed=H, fill=0.0)
    want, want_lse = ref.paged_mla(q, cache, table, lens, cu, D ** -0.5, page)
    q[0], q[4, 0] = float("nan"), INF
    out, lse = run(q, cache, table, lens, cu, D)
    keep = torch.ones(6, H, dtype=torch.bool)
    keep[0], keep[4, 0] = False, False
    check(out[keep], want[keep], lse[keep], want_lse[keep])
    assert bool(out[~keep].isnan().all())
