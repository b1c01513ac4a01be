"""dsa_norm_rope_fwd with cache rows that several tokens name: every channel of such a row is that of one of them."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("D,norm_dim", [(576, 512), (128, 128), (97, 97)])
def test_a_row_named_twice_gets_each_channel_from_one_of_the_results(D, norm_dim):
    T, rows = 900, 40
    g = torch.Generator().manual_seed(D)
    x = torch.randn(T, D, generator=g).bfloat16().to(DEV)
    pos = torch.randint(0, 5000, (T,), generator=g).to(torch.int32).to(DEV)
    f = dsa.dsa_rope_frequencies(32)[0]
    kw = dict(inv_freq=f, positions=pos, norm="rms", norm_dim=norm_dim, rope_start=0)
    each = dsa.dsa_norm_rope_fwd(x, **kw)
    to = torch.randint(-1, rows // 2, (T,), generator=g).to(torch.int32)
    cache = torch.full((rows, D), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    dsa.dsa_norm_rope_fwd(x, out=cache, out_rows=to.to(DEV), workspace=ws, **kw)
    for r in range(rows):
        mine = each[(to == r).to(DEV)]
        assert bool((mine == cache[r]).any(0).all()) if len(mine) else bool((cache[r] == 7).all())
    assert dsa.dsa_read_device_status(ws) == 0
