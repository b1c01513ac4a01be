"""dsa_norm_rope_fwd / bwd with values that are not finite: they reach their pair of rotated channels (and, under the norm,
what the norm covers), and no channel else.  Channels that are neither normalised nor rotated are copied, the sign of a
zero included.  And values at both ends of what a norm takes (|x| < 2^57; above 2^-58 with eps = 0): tolerances of
test_gpu_norm_rope.py, which follow the rows' own magnitudes."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref
from test_gpu_norm_rope import f64, near, near_sum

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, H = 40, 3

CASES = [  # D, norm_dim, R, r0, interleaved, wide
    (192, 0, 64, 128, False, 0),
    (192, 0, 64, 128, True, 0),
    (128, 0, 64, 0, False, 0),
    (128, 0, 64, 0, True, 0),
    (64, 0, 32, 16, False, 0),
    (64, 0, 16, 48, True, 8),
    (256, 0, 128, 64, False, 0),
    (576, 512, 64, 512, True, 0),
    (576, 512, 64, 512, False, 0),
    (192, 128, 64, 128, False, 0),
    (192, 128, 32, 160, True, 0),
    (1024, 0, 256, 256, False, 0),
    (1024, 0, 64, 40, True, 0),
    (128, 0, 48, 4, False, 0),       # rotated channels that start inside an access
    (97, 0, 30, 67, True, 0),        # one channel at a time
    (97, 0, 30, 11, False, 1),
]


def partner(c, R, r0, inter):
    u = c - r0
    return r0 + ((u ^ 1) if inter else (u + R // 2) % R)


@pytest.mark.parametrize("D,n,R,r0,inter,wide", CASES)
@pytest.mark.parametrize("back", [False, True])
def test_values_reach_their_pair_only(D, n, R, r0, inter, wide, back):
    g = torch.Generator().manual_seed(D + R + r0)
    clean = torch.randn(T, H, D + wide, generator=g).bfloat16()
    pos = torch.randint(0, 5000, (T,), generator=g).to(torch.int32).to(DEV)
    f = torch.tensor([10000.0 ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float32, device=DEV)
    plain = [c for c in range(n, D) if not r0 <= c < r0 + R]  # channels that are copied
    clean[:, :, [wide + c for c in plain[::3]]] = -0.0
    bad = clean.clone()
    touched = torch.zeros(T, H, D, dtype=torch.bool)
    values = [float("inf"), -float("inf"), float("nan")]
    for t in range(T):
        for h in range(H):
            v = values[(t + h) % 3]
            c = r0 + int(torch.randint(0, R, (1,), generator=g))
            bad[t, h, wide + c] = v
            touched[t, h, [c, partner(c, R, r0, inter)]] = True
            if plain:  # neighbours of both layouts among them, over the rows
                c = plain[int(torch.randint(0, len(plain), (1,), generator=g))]
                bad[t, h, wide + c] = v
                touched[t, h, c] = True
    kw = dict(inv_freq=f, positions=pos, norm="rms" if n else "none", norm_dim=n, rope_start=r0, interleaved=inter)
    x = torch.randn(T, H, D, generator=g).bfloat16().to(DEV)

    def call(v):
        v = v.to(DEV)[..., wide:]
        return (dsa.dsa_norm_rope_bwd(v, x if n else None, **kw)[0] if back else dsa.dsa_norm_rope_fwd(v, **kw)).cpu()

    want, got = call(clean), call(bad)
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(got)[~touched], bits(want)[~touched])
    if plain:
        a, b = bad[..., wide:][..., plain], got[..., plain]
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(bits(a)[~a.isnan()], bits(b)[~a.isnan()])
        assert torch.equal(bits(clean[..., wide:][..., plain]), bits(want[..., plain]))
    rot = got[..., r0:r0 + R]
    assert not bool(rot[touched[..., r0:r0 + R]].isfinite().any())  # (0 times an infinity is NaN)


@pytest.mark.parametrize("kind,n,D", [("rms", 512, 576), ("layer", 128, 128), ("rms", 97, 97), ("layer", 1024, 1024)])
@pytest.mark.parametrize("power", [54, -56])
def test_the_largest_and_smallest_rows_of_a_norm(kind, n, D, power):
    g = torch.Generator().manual_seed(n)
    x = (torch.randn(20, 2, D, generator=g).clamp(-7, 7) * 2.0 ** power).bfloat16().to(DEV)
    x[..., 0] = 7.5 * 2.0 ** power
    dout = torch.randn(20, 2, D, generator=g).bfloat16().to(DEV)
    w = (1 + 0.3 * torch.randn(n, generator=g)).to(DEV)
    kw = dict(norm=kind, norm_dim=n, weight=w, eps=0.0)
    none = (None, None, D, False)
    y = dsa.dsa_norm_rope_fwd(x, **kw)
    near(y[..., :n], ref.norm_rope_fwd(f64(x), kind, n, f64(w), None, 0.0, *none)[..., :n], "y")
    assert torch.equal(y[..., n:], x[..., n:])
    dx, dw, _ = dsa.dsa_norm_rope_bwd(dout, x, **kw)
    # (a gradient is as much smaller as its row is larger: compared with that of the rows at ordinary size)
    rdx, rdw, _, mw, _, most = ref.norm_rope_bwd(f64(dout), f64(x) / 2.0 ** power, kind, n, f64(w), 0.0, *none)
    near(dx.double()[..., :n] * 2.0 ** power, rdx[..., :n], "dx", most)
    assert torch.equal(dx[..., n:], dout[..., n:])
    near_sum(dw, rdw, mw, "dw")
