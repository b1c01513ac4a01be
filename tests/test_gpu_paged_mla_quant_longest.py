"""Attention over the longest request that a quantised cache can hold: its output."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _quant_ref as ref
from test_gpu_paged_mla_quant import workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("scale", [0.04, 0.5])
def test_the_output_of_the_longest_request(bits, scale):
    """2^31 - 1 positions in one page of 64 that the table names again and again: the output of those 64 (that one position of
    2^25 rounds of them is missing is nothing beside the sums).  Every CTA adds 6 products of each of its tiles of 64 (or
    fewer, of 96) one after the other: 6 * 2^25 / 152 additions, each off by 2^-23 of the mass at most, by truncation too, and
    the sum of weights fewer than that; then the weights' and the output's own rounding.  With the larger scale one row has
    most of the mass, so that the tolerance is a sixth of the output's channels."""
    g = torch.Generator().manual_seed(5)
    cache = torch.zeros(1, 64, dsa.paged_quant_row_bytes(512, bits), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(torch.randn(64, 512, generator=g).bfloat16().to(DEV), cache, bits)
    q = torch.randn(1, 1, 512, generator=g).bfloat16()
    ws = workspace()
    lens = torch.tensor([2 ** 31 - 1], dtype=I32, device=DEV)
    out, _ = dsa.dsa_paged_mla_quant(q.to(DEV), cache, torch.zeros(1, 2 ** 25, dtype=I32, device=DEV), lens, scale, bits,
                                     workspace=ws)
    want, _, size, mass, _, most = ref.attention(q, cache, bits, torch.zeros(1, 1, dtype=I32), [64], [0, 1], scale)
    dz = 84 * 2.0 ** -23 * size + 2.0 ** -20 + (2.0 ** -17 * most if bits == 8 else 0.0)
    tol = 2.0 ** -8 * want.abs() + (6 * 2 ** 25 / 152 * 2.0 ** -23 + 2.0 ** -10 + 2 * dz)[..., None] * mass
    off = (out.cpu().double() - want).abs()
    assert dsa.dsa_read_device_status(ws) == 0
    assert float((want.abs() > tol).double().mean()) > (0.9 if scale > 0.1 else 0.2)
    assert bool((off <= tol).all()), float((off / tol).max())
    print("off / mass", float((off / mass).max()))
