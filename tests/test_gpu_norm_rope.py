"""dsa_norm_rope_fwd / bwd against the 64-bit definitions.

Tolerances.  A stored row is rounded once to bf16: half a step, 2^-8 of the value.  Before that everything is fp32:
the statistics are sums of at most 1024 terms (relative error below 1024 * 2^-24 = 2^-14 in the worst order), the
angle is off by at most 2^-24 half turns and the sine and cosine by a few 2^-24, so a value is off by at most 2^-13
of the largest magnitude of its row.  dx is r gw - r xh mean(gw xh) (- r mean gw), and these terms may cancel (one
channel: gw (1 - xh^2) with xh near 1): each of them is off by 2^-13 of itself, so dx by 2^-13 of the terms' sum, and
not of what is left of it.  A sum over rows (dweight, dbias) is formed in fp32 from such terms: at most
2^-13 of the sum of the magnitudes of its terms."""
import numpy as np
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def near(got, want, what, most=None):
    got = f64(got)
    most = np.abs(want).max(-1, keepdims=True) if most is None else most
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -13 * most + 1e-30
    assert np.all(np.abs(got - want) <= bound), f"{what}: {np.max(np.abs(got - want) / bound)}"


def near_sum(got, want, terms, what):
    assert np.all(np.abs(f64(got) - want) <= 2.0 ** -13 * terms + 1e-30), what


def inputs(T, H, D, kind, n, R, seed, far=100000, wide=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D + wide, generator=g).bfloat16().to(DEV)[..., wide:]
    dout = torch.randn(T, H, D + wide, generator=g).bfloat16().to(DEV)[..., wide:]
    w = (1 + 0.3 * torch.randn(n, generator=g)).to(DEV) if kind != "none" else None
    b = (0.3 * torch.randn(n, generator=g)).to(DEV) if kind == "layer" else None
    pos = torch.randint(0, far, (T,), generator=g).to(torch.int32).to(DEV)
    f = dsa.dsa_rope_frequencies(R)[0] if R else None
    return x, dout, w, b, pos, f


CASES = [  # T, H, D, norm, n, R, r0, interleaved, wide
    (5, 1, 576, "rms", 512, 64, 512, True, 0),
    (1, 1, 576, "rms", 512, 64, 512, False, 0),
    (300, 1, 128, "layer", 128, 64, 0, False, 0),
    (37, 3, 128, "rms", 128, 128, 0, True, 0),
    (700, 40, 64, "none", 0, 64, 0, True, 512),
    (41, 24, 192, "none", 0, 64, 128, False, 8),
    (9, 2, 97, "layer", 97, 30, 67, True, 0),
    (9, 2, 97, "rms", 50, 30, 11, True, 1),
    (33, 5, 80, "layer", 80, 40, 8, False, 0),
    (10, 1, 1024, "layer", 1024, 1024, 0, False, 0),
    (6, 2, 1000, "rms", 999, 2, 998, True, 3),
    (50, 2, 256, "rms", 200, 16, 3, False, 0),
    (64, 1, 512, "rms", 512, 0, 512, False, 0),
    (7, 1, 1, "rms", 1, 0, 1, False, 0),
    (3, 2, 700, "layer", 640, 60, 640, True, 4),
]


@pytest.mark.parametrize("T,H,D,kind,n,R,r0,inter,wide", CASES)
def test_forward_and_gradient(T, H, D, kind, n, R, r0, inter, wide):
    x, dout, w, b, pos, f = inputs(T, H, D, kind, n, R, seed=T + D, wide=wide)
    eps, scale = 1e-5, 1.25 if R else 1.0
    ws = torch.zeros(dsa.paged_workspace_size("norm_rope_bwd", T * H, n), dtype=torch.uint8, device=DEV)
    kw = dict(inv_freq=f, positions=pos, norm=kind, norm_dim=n, weight=w, eps=eps, rope_start=r0, interleaved=inter,
              rope_scale=scale, workspace=ws)
    y = dsa.dsa_norm_rope_fwd(x, bias=b, **kw)
    assert y.shape == x.shape
    near(y, ref.norm_rope_fwd(f64(x), kind, n, f64(w), f64(b), eps, f64(pos), f64(f), r0, inter, scale), "y")
    dx, dw, db = dsa.dsa_norm_rope_bwd(dout, x, with_bias=kind == "layer", **kw)
    rdx, rdw, rdb, mw, mb, most = ref.norm_rope_bwd(f64(dout), f64(x), kind, n, f64(w), eps, f64(pos), f64(f), r0, inter, scale)
    near(dx, rdx, "dx", most)
    if kind != "none":
        near_sum(dw, rdw, mw, "dw")
    if kind == "layer":
        near_sum(db, rdb, mb, "db")
    assert dsa.dsa_read_device_status(ws) == 0
    # the same call again gives the same bits, and accumulate adds
    dx2, dw2, db2 = dsa.dsa_norm_rope_bwd(dout, x, with_bias=kind == "layer", **kw)
    assert torch.equal(dx, dx2) and (dw is None or torch.equal(dw, dw2)) and (db is None or torch.equal(db, db2))
    if kind != "none":
        dsa.dsa_norm_rope_bwd(dout, x, with_bias=kind == "layer", dweight=dw2, dbias=db2, accumulate=True, **kw)
        assert torch.equal(dw2, dw + dw) and (db is None or torch.equal(db2, db + db))


@pytest.mark.parametrize("far", [10, 2 ** 20, 2 ** 31 - 1])
def test_far_and_negative_positions(far):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(64, 1, 64, generator=g).bfloat16().to(DEV)
    pos = (torch.randint(0, far, (64,), generator=g)).to(torch.int32)
    pos[1::2] *= -1
    pos[0] = -2 ** 31 if far > 2 ** 30 else 0
    f = torch.tensor([7.5, 1.0, 0.3] + [10000.0 ** (-i / 32) for i in range(29)], dtype=torch.float32)
    y = dsa.dsa_norm_rope_fwd(x, inv_freq=f.to(DEV), positions=pos.to(DEV))
    near(y, ref.norm_rope_fwd(f64(x), "none", 0, None, None, 0, f64(pos), f64(f), 0, False), "y")


def test_in_place_and_strided_rows():
    x, dout, w, b, pos, f = inputs(50, 6, 64, "none", 0, 64, seed=3)
    q = torch.randn(50, 6, 576, device=DEV).bfloat16()
    q[..., 512:] = x
    keep = q[..., :512].clone()
    want = dsa.dsa_norm_rope_fwd(x, inv_freq=f, positions=pos)
    view = q[..., 512:]
    assert dsa.dsa_norm_rope_fwd(view, inv_freq=f, positions=pos, out=view) is view
    assert torch.equal(q[..., 512:], want) and torch.equal(q[..., :512], keep)
    # heads before tokens
    xt = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(dsa.dsa_norm_rope_fwd(xt, inv_freq=f, positions=pos, out=torch.empty_like(xt)), want)
    # a row that all heads share (stride 0)
    one = dsa.dsa_norm_rope_fwd(x[:, :1].expand(50, 6, 64), inv_freq=f, positions=pos, out=torch.empty_like(x))
    assert torch.equal(one, want[:, :1].expand(50, 6, 64))
    # the gradient into its own storage
    dx, _, _ = dsa.dsa_norm_rope_bwd(dout.clone(), inv_freq=f, positions=pos)
    d2 = dout.clone()
    dsa.dsa_norm_rope_bwd(d2, inv_freq=f, positions=pos, dx=d2)
    assert torch.equal(dx, d2)


def test_rows_go_to_their_slots_and_no_other():
    T, P = 70, 16
    x, _, w, _, pos, f = inputs(T, 1, 576, "rms", 512, 64, seed=5)
    kw = dict(inv_freq=f, positions=pos, norm="rms", norm_dim=512, weight=w, interleaved=True)
    want = dsa.dsa_norm_rope_fwd(x[:, 0], **kw)
    cache = torch.full((12, P, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    slots = torch.randperm(12 * P)[:T].to(torch.int32)
    slots[[3, 40]] = -1
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    dsa.dsa_norm_rope_fwd(x[:, 0], out=cache, out_rows=slots.to(DEV), workspace=ws, **kw)
    flat = cache.view(-1, 576)
    expect = torch.full_like(flat, 7.0)
    keep = slots >= 0
    expect[slots[keep].long().to(DEV)] = want[keep.to(DEV)]
    assert torch.equal(flat, expect) and dsa.dsa_read_device_status(ws) == 0
    # rows outside the cache are skipped and reported
    slots[5], slots[6] = 12 * P, -2
    before = cache.clone()
    dsa.dsa_norm_rope_fwd(x[:, 0], out=cache, out_rows=slots.to(DEV), workspace=ws, **kw)
    assert torch.equal(cache, before) and dsa.dsa_read_device_status(ws) == 6


def test_values_that_are_not_finite_stay_in_their_row():
    x, dout, w, b, pos, f = inputs(64, 1, 128, "layer", 128, 64, seed=8)
    kw = dict(inv_freq=f, positions=pos, norm="layer", weight=w, rope_start=0)
    want = dsa.dsa_norm_rope_fwd(x, bias=b, **kw)
    x2 = x.clone()
    x2[7, 0, 3], x2[20, 0, 100] = float("nan"), float("inf")
    got = dsa.dsa_norm_rope_fwd(x2, bias=b, **kw)
    ok = [i for i in range(64) if i not in (7, 20)]
    assert torch.equal(got[ok], want[ok]) and bool(got[7].isnan().all()) and bool(got[20].isnan().any())


def test_no_rows():
    f = dsa.dsa_rope_frequencies(64)[0]
    e = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    pos = torch.empty(0, dtype=torch.int32, device=DEV)
    assert dsa.dsa_norm_rope_fwd(e, inv_freq=f, positions=pos).shape == (0, 2, 128)
    dx, dw, db = dsa.dsa_norm_rope_bwd(e, e, inv_freq=f, positions=pos, norm="layer", with_bias=True)
    assert dx.shape == (0, 2, 128) and bool((dw == 0).all()) and bool((db == 0).all())


def test_another_stream_and_a_captured_backward():
    x, dout, w, b, pos, f = inputs(200, 4, 128, "rms", 128, 128, seed=11)
    kw = dict(inv_freq=f, positions=pos, norm="rms", weight=w, rope_start=0)
    dx, dw, _ = dsa.dsa_norm_rope_bwd(dout, x, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        dx2, dw2, _ = dsa.dsa_norm_rope_bwd(dout, x, **kw)
    s.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dx3, dw3, _ = dsa.dsa_norm_rope_bwd(dout, x, **kw)
    for _ in range(2):
        dx3.zero_(), dw3.zero_()
        g.replay()
        assert torch.equal(dx, dx3) and torch.equal(dw, dw3)
