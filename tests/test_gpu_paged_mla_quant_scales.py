"""Attention over quantised rows whose scales differ by up to 2^60 while their scores stay within a few tens, so that every
head has rows of one size that carry its output: with a tolerance that is a small part of it."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _quant_ref as ref
from test_gpu_paged_mla_quant import make, run, workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SIZES = (-30, -18, -6, 6, 18, 30)
WIDTH = 80  # channels of a kind of rows
SCALE = 0.125


def rows_and_queries(H, lens, news, g):
    """Rows of six kinds: kind c has 80 latent channels of its own, of size 2^SIZES[c], and position channel c.  Head h
    prefers the rows of kind h % 6 by 60 nats, and among them by their latents, by about 2."""
    x = torch.zeros(sum(lens), 576)
    kind = torch.randint(0, 6, (len(x),), generator=g)
    kind[:6 * len(lens)] = torch.arange(6).repeat(len(lens))
    x[:, 520:] = 0.5 * torch.randn(len(x), 56, generator=g)
    for c, e in enumerate(SIZES):
        own = kind == c
        x[own, c * WIDTH:(c + 1) * WIDTH] = torch.randn(int(own.sum()), WIDTH, generator=g) * 2.0 ** e
        x[own, 512 + c] = 1
    q = torch.zeros(sum(news), H, 576)
    q[..., 520:] = 0.5 * torch.randn(sum(news), H, 56, generator=g)
    for h in range(H):
        c = h % 6
        q[:, h, 512 + c] = 480
        q[:, h, c * WIDTH:(c + 1) * WIDTH] = torch.randn(sum(news), WIDTH, generator=g) * (2 / SCALE / WIDTH ** 0.5 * 2.0 ** -SIZES[c])
    return x.bfloat16(), q.bfloat16()


def expect(q, rows, bits):
    """out, lse and their tolerances [H, 512], [H] of one token that sees these rows.  As in check_attention and
    check_closely of the other tests, but with the error of a score by position: 84 * 2^-23 of its sum of magnitudes, and with 8
    bits 2^-17 of the query row's largest channel for each latent channel that is not zero."""
    kv = ref.decode(rows, 576, 512, bits)
    q = q.double()
    z = q @ kv.T * SCALE
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    dz = 84 * 2.0 ** -23 * SCALE * (q.abs() @ kv.abs().T) + 2.0 ** -20
    if bits == 8:
        lat = q[:, :512]
        dz = dz + 2.0 ** -17 * SCALE * lat.abs().amax(1, keepdim=True) * ((lat != 0).double() @ kv[:, :512].abs().T)
    v, mean = kv[:, :512], (p * dz).sum(1)
    mass = p @ v.abs()
    at = ref.layout(576, 512, bits)[1]
    s = rows[:, at:at + 4].contiguous().view(torch.float32).double()
    top = (p * s[:, 0]).amax(1, keepdim=True) * (v.abs() / s).sum(0)
    tol = 2.0 ** -8 * (p @ v).abs() + 2 * ((p * dz) @ v.abs()) + (2.0 ** -11 + 2.0 ** -13 + 2 * mean)[:, None] * mass
    tol = tol + (2.0 ** -28 if bits == 8 else 2.0 ** -32) * top
    return p @ v, lse, tol, mean + 2.0 ** -13 + 2.0 ** -22 * lse.abs(), mass


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H", [16, 64])
def test_rows_whose_scales_differ_by_far(bits, H):
    lens, news = [500, 129], [1, 3]
    g, cache, table, _, cu = make(bits, 576, H, 64, lens, news, 3)
    x, q = rows_and_queries(H, lens, news, g)
    slots = [[int(table[b, p // 64]) * 64 + p % 64 for p in range(n)] for b, n in enumerate(lens)]
    dsa.dsa_paged_quantize(x.to(DEV), cache, bits, out_rows=torch.tensor(sum(slots, []), dtype=torch.int32, device=DEV))
    ws = workspace()
    out, lse = run(bits, cache, table, q, lens, cu, SCALE, ws=ws)
    assert dsa.dsa_read_device_status(ws) == 0
    flat = cache.cpu().view(-1, cache.shape[2])
    own = torch.stack([(torch.arange(512) // WIDTH) == h % 6 for h in range(H)])
    for b in range(2):
        for n in range(cu[b], cu[b + 1]):
            seen = lens[b] - news[b] + n - cu[b] + 1
            want, l, tol, l_tol, mass = expect(q[n], flat[slots[b][:seen]], bits)
            # (in the channels of a head's own rows an output of zeros would not pass)
            assert bool((tol <= 0.02 * mass)[own].all()) and float((want.abs() > tol)[own].double().mean()) > 0.9
            assert bool(((lse[n].cpu().double() - l).abs() <= l_tol).all())
            off = (out[n].cpu().double() - want).abs()
            assert bool((off <= tol).all()), float((off / tol).max())
