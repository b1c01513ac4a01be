"""Attention over a quantised cache where one position is far above the others and the others carry the output all the same:
many of them, equal or nearly so, so that what each weight is off by adds up.  The output's error is held against the output
(and the mass of what was added), not against the number of positions times the largest weight."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _quant_ref as ref
from test_gpu_paged_mla_quant import run, workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def check_closely(got, want, bits, n):
    """out and lse for requests of n positions at most, against ref.attention()'s answer.

    Scores: as in ref.check_attention.  A weight: three numbers of 3 bits (8 bits: half a step of the first is 2^-3 of the
    weight's power of two 2^E; what it leaves is below 2^(E-3), so that half a step of the second is 2^(E-7), and of the third
    2^(E-11)) or one of 11 (4 bits): 2^-11 of the weight.  Where the steps of the type end: multiples of 2^-16 (8 bits; the
    largest weight times its row's s is 2^11 at least) or 2^-24 (4 bits; 2^7), half a step being 2^-28 or 2^-32 of the largest.

    Sums: 6 products of a tile of 64 positions (or fewer, of 96) are added one after the other, each of them a sum of 16 or 32,
    and each addition is off by 2^-23 of the mass at most, by truncation too, and the sum within the product by as much.
    A thread's sum of weights has fewer terms.  The output is rounded to bf16."""
    out, lse, size, mass, top, most = want
    o, l = got[0].cpu().double(), got[1].cpu().double()
    sums = 2 * 6 * (n / 64 + 1) * 2.0 ** -23
    dz = 84 * 2.0 ** -23 * size + 2.0 ** -20 + (2.0 ** -17 * most if bits == 8 else 0.0)
    assert bool(((l - lse).abs() <= dz + sums + 2.0 ** -22 * lse.abs()).all()), float(((l - lse).abs() - dz).max())
    floor = 2.0 ** -28 if bits == 8 else 2.0 ** -32
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2 * sums + 2 * dz)[..., None] * mass + floor * top + 2.0 ** -133
    # (a tolerance that lets anything pass would show nothing)
    assert bool((tol <= 0.1 * mass).double().mean() > 0.5)
    assert bool((o - out).abs().le(tol).all()), float(((o - out).abs() / tol).max())


@pytest.mark.parametrize("n", [16384, 131072])
@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("bits", [8, 4])
def test_many_positions_far_below_the_first(bits, H, n):
    """160 requests over the same pages, so that a CTA has whole requests; the first position is 5 to 11 nats above the
    others, which are equal (even heads) or spread by 0.3 nats, with values that have a common mean."""
    g = torch.Generator().manual_seed(n + H)
    page, B = 64, 160
    x = torch.zeros(n, 576)
    x[:, :512] = 1 + 0.25 * torch.randn(n, 512, generator=g)
    x[0, :512] -= 2
    x[0, 512] = 1
    x[1:, 513] = 0.3 * torch.randn(n - 1, generator=g)
    cache = torch.zeros(n // page, page, dsa.paged_quant_row_bytes(576, bits), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(x.bfloat16().to(DEV), cache, bits)
    table = torch.arange(n // page, dtype=I32)[None]
    q = torch.zeros(1, H, 576)
    q[0, :, 512] = 5 + 6 * torch.arange(H) / (H - 1)
    q[0, 1::2, 513] = 1
    q = q.bfloat16()
    ws = workspace()
    out, lse = run(bits, cache, table.repeat(B, 1), q.repeat(B, 1, 1), [n] * B, list(range(B + 1)), 1.0, ws=ws)
    assert dsa.dsa_read_device_status(ws) == 0
    check_closely((out, lse), ref.attention(q, cache, bits, table, [n], [0, 1], 1.0), bits, n)


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("bits", [8, 4])
def test_a_small_weight_keeps_its_bits(bits, H, listed):
    """Two positions, the second 2^0 to 2^-20 of the first by head, each with values in channels of its own; in one tile,
    and in tiles of their own."""
    g = torch.Generator().manual_seed(H)
    x = torch.zeros(16, 576)
    x[0, :256] = torch.rand(256, generator=g) + 1
    x[1, 256:512] = torch.rand(256, generator=g) + 1
    x[0, 512] = 1
    cache = torch.zeros(1, 16, dsa.paged_quant_row_bytes(576, bits), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(x.bfloat16().to(DEV), cache, bits)
    table = torch.zeros(1, 1, dtype=I32)
    q = torch.zeros(1, H, 576)
    q[0, :, 512] = 20 * torch.arange(H) / (H - 1)
    q = q.bfloat16()
    scale = float(torch.tensor(2.0).log())
    idx = None
    if listed:
        idx = torch.full((1, 200), -1, dtype=I32)
        idx[0, 0], idx[0, 199] = 0, 1
    B = 400  # (the same request many times, so that a CTA has whole ones)
    got = run(bits, cache, table.repeat(B, 1), q.repeat(B, 1, 1), [2] * B, list(range(B + 1)), scale,
              idx.repeat(B, 1) if listed else None)
    check_closely(got, ref.attention(q, cache, bits, table, [2], [0, 1], scale, None, idx), bits, 200)
