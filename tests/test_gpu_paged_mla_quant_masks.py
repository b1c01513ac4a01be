"""Attention over a quantised cache whose tables have holes: rows are masked in one tile and live in the next at the same
place, so that what lies in a masked row's place is a live row of the tile before.  Few rows of a request are live: one that
is dropped, or one too many, moves the output by far more than its tolerance."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _quant_ref as ref
from test_gpu_paged_mla_quant import make, run, workspace

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("page,live", [(16, 5), (32, 3), (64, 2), (7, 9)])
def test_pages_that_are_missing_between_others(bits, H, page, live):
    """60 requests of 1500 to 2090 positions: several tiles for each CTA."""
    lens = [1500 + 10 * b for b in range(60)]
    g, cache, table, q, cu = make(bits, 576, H, page, lens, [1] * 60, page)
    holes, keep = table.clone(), torch.full((60, live * page), -1, dtype=I32)
    for b, n in enumerate(lens):
        pages = -(-n // page)
        there = torch.randperm(pages, generator=g)[:live].sort().values
        gone = torch.ones(pages, dtype=torch.bool)
        gone[there] = False
        values = torch.tensor([-1, cache.shape[0], -2 ** 31, 2 ** 31 - 1], dtype=I32)
        holes[b, :pages][gone] = values[torch.randint(0, 4, (int(gone.sum()),), generator=g)]
        at = [p for c in there.tolist() for p in range(c * page, min(n, (c + 1) * page))]
        keep[b, :len(at)] = torch.tensor(at, dtype=I32)
    ws = workspace()
    want = ref.attention(q, cache, bits, table, lens, cu, 0.02, topk=keep)
    for _ in range(3):
        got = run(bits, cache, holes, q, lens, cu, 0.02, ws=ws)
        assert dsa.dsa_read_device_status(ws) == 6
        ref.check_attention(got, want, bits)
