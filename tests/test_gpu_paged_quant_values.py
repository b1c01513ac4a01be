"""Rows of a quantised cache: every bf16 magnitude is written as the format says."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _quant_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("top", [1.3125 * 2.0 ** 20, 1.7578125 * 2.0 ** 3, 1.75 * 2.0 ** 56, 1.5 * 2.0 ** -38])
def test_all_magnitudes_of_bf16_below_the_largest(bits, top):
    """Each of them, of both signs, in a block of 16 where it lies beside the row's largest magnitude and in one of its like."""
    mags = torch.arange(0, 0x7f80, dtype=torch.int16).view(torch.bfloat16)
    v = mags[mags.double() <= top]
    v = torch.cat([v, torch.zeros(-len(v) % 62, dtype=torch.bfloat16)]).reshape(-1, 62)
    x = torch.cat([torch.full((len(v), 1), top, dtype=torch.bfloat16), v, torch.zeros(len(v), 9, dtype=torch.bfloat16)], 1)
    x = torch.cat([x, -x])
    assert bool((x[:, 0].double().abs() == top).all())
    c = torch.zeros(len(x), dsa.paged_quant_row_bytes(72, bits, 64), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(x.to(DEV), c, bits, 64)
    assert torch.equal(c.cpu(), ref.encode(x, 64, bits))
