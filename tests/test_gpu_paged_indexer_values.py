"""dsa_paged_indexer_topk over keys with infinities: a key's score is the sum over its token's heads and nothing else, whatever
number of heads the kernel works on at once.  Scores and lists by the definition in 64 bits; the values lie on a grid on which
every finite sum is exact in fp32 (multiples of 1/8 up to 3, weights that are multiples of 1/1024), so the lists have to be equal."""
import pytest
import torch

import _paged_ref as ref
from test_gpu_paged_indexer import make, run

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("Hi", [1, 3, 5, 7, 8, 9, 12, 16, 20, 31, 32, 33, 40, 63, 64])
@pytest.mark.parametrize("page", [64, 33])
def test_infinite_keys(Hi, page):
    lens, news, K = [700, 150], [3, 2], 60
    q, k, w, table, cu = make(lens, news, Hi, page, seed=Hi)
    w = (w.abs() * 1024).round().clamp(min=1) / 1024
    q[..., 0], q[..., 1], q[..., 2] = 1.0, -0.5, -2.0
    q[:, 0, 2] = 0.25  # of channel 2 one head's product is positive
    flat = k.view(-1, 128)
    for b, n in enumerate(lens):
        rows = ref.rows_of(table[b], range(n), page)
        for at, channel, value in ((5, 0, INF), (40, 0, -INF), (77, 1, INF), (90, 1, -INF), (101, 2, INF), (n - 2, 0, -INF),
                                   (n - 1, 2, INF)):
            flat[rows[at], channel] = value
    idx, ln = run(q, k, w, table, lens, cu, K)
    for b in range(2):
        for n in range(cu[b], cu[b + 1]):
            v = ref.visible(lens[b], news[b], n - cu[b])
            s = ref.paged_scores(q[n], k, w[n], table[b], v, page)[0]
            assert not bool(s.isnan().any()) and int(torch.isinf(s).sum()) == 4 - (v < lens[b])
            want = ref.topk_of(s, K)
            assert ln[n] == K and idx[n].tolist() == want, (b, n)
