"""The serving calls over batches and lists without entries."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def ints(*shape):
    return torch.zeros(*shape, dtype=I32, device=DEV)


def test_lists_without_columns_are_refused():
    # they name no position; without a column they have no address, and were answered like no lists: with all positions
    q = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="topk_idx"):
        dsa.dsa_paged_mla(q, cache, ints(2, 1), torch.ones(2, dtype=I32, device=DEV), 0.1, topk_idx=ints(2, 0))
    # entries of -1 are how a list says so
    sink = torch.linspace(-1, 1, 16, device=DEV)
    none = torch.full((2, 1), -1, dtype=I32, device=DEV)
    out, lse = dsa.dsa_paged_mla(q, cache, ints(2, 1), torch.ones(2, dtype=I32, device=DEV), 0.1, topk_idx=none, attn_sink=sink)
    assert bool((out == 0).all()) and bool(((lse - sink).abs() <= 2.0 ** -22).all())


@pytest.mark.parametrize("B", [0, 3])  # no requests; requests without new tokens
@pytest.mark.parametrize("with_len", [False, True])
def test_lists_of_no_tokens(B, with_len):
    cache = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device=DEV)
    keys = torch.zeros(2, 16, 128, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(0, 16, 576, dtype=torch.bfloat16, device=DEV)
    qi = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device=DEV)
    table, lens, cu = ints(B, 2), ints(B), ints(B + 1)
    idx, n = dsa.dsa_paged_indexer_topk(qi, keys, torch.zeros(0, 8, device=DEV), table, lens, 20, cu_q=cu)
    assert idx.shape == (0, 20) and n.shape == (0,)
    out, lse = dsa.dsa_paged_mla(q, cache, table, lens, 0.1, cu_q=cu, topk_idx=idx, topk_len=n if with_len else None)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
    torch.cuda.synchronize()
