"""Queries over a quantised cache whose channels are of very different size."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _quant_ref as ref
from test_gpu_paged_mla_quant import make, run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("large", [29, 41, 53])
def test_a_query_with_one_large_position_channel(bits, H, large):
    """Of size 2^large beside latent channels of size 1, where the keys' channel is zero.  4 bits: a query's latent channels
    count to a multiple of 2^-24 of what takes 2^-24 of the row's largest channel to 2^14 at least, which is off by 2^-63 of
    that channel at most; 8 bits: the position channels do not enter into it."""
    lens = [400, 200]
    g, cache, table, _, cu = make(bits, 576, H, 64, lens, [1, 1], large)
    x = torch.randn(600, 576, generator=g)
    x[:, 515] = 0
    slots = [[int(table[b, p // 64]) * 64 + p % 64 for p in range(n)] for b, n in enumerate(lens)]
    dsa.dsa_paged_quantize(x.bfloat16().to(DEV), cache, bits, out_rows=torch.tensor(sum(slots, []), dtype=torch.int32, device=DEV))
    q = torch.randn(2, H, 576, generator=g)
    q[..., 515] = 2.0 ** large
    q = q.bfloat16()
    out, lse = run(bits, cache, table, q, lens, cu, 0.05)
    want = list(ref.attention(q, cache, bits, table, lens, cu, 0.05))
    # (size bounds dz through 84 * 2^-23 size: the loss of the query's channels is added to it)
    if bits == 4:
        lost = 2.0 ** (large - 63) * want[5] / q[..., :512].double().abs().amax(2)
        want[2] = want[2] + lost * 2.0 ** 23 / 84
        assert float(lost.max()) < 0.5
    ref.check_attention((out, lse), tuple(want), bits)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [16, 64])
def test_rows_and_queries_of_position_channels_alone(bits, H):
    """Every second row has latents of zero, and so the least s; of the queries every second head has, and every third head
    latents that are 2^-30 of its position channels."""
    lens = [400, 200]
    g, cache, table, _, cu = make(bits, 576, H, 64, lens, [1, 1], H)
    x = torch.randn(600, 576, generator=g)
    x[:, 512:] *= 64
    x[::2, :512] = 0
    slots = [[int(table[b, p // 64]) * 64 + p % 64 for p in range(n)] for b, n in enumerate(lens)]
    dsa.dsa_paged_quantize(x.bfloat16().to(DEV), cache, bits, out_rows=torch.tensor(sum(slots, []), dtype=torch.int32, device=DEV))
    q = torch.randn(2, H, 576, generator=g)
    q[:, ::3, :512] *= 2.0 ** -30
    q[:, ::2, :512] = 0
    q = q.bfloat16()
    got = run(bits, cache, table, q, lens, cu, 0.01)
    ref.check_attention(got, ref.attention(q, cache, bits, table, lens, cu, 0.01), bits)
