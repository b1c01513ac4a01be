"""CPU checks of the serving step's entry points: what the library and the binding refuse before anything is launched,
the frequency table, and the tests' own gradient formulas against differences."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_attention_mla_gb300 as dsa
from sparse_attention_mla_gb300 import build_ext

import _paged_ref as ref

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: validation fails before any device use
WS = P(0x100000)


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return dsa.load_library()


def test_names_and_status(lib):
    for name in ("dsa_paged_slots", "dsa_norm_rope_fwd", "dsa_norm_rope_bwd", "dsa_rope_frequencies", "dsa_paged_mla",
                 "dsa_paged_indexer_topk"):
        assert callable(getattr(dsa, name)) and name in dsa.declared_symbols() and hasattr(lib, name)
    assert lib.dsa_status_string(8).decode().startswith(dsa.STATUS_NAMES[8])


def slots(lib, **kw):
    a = dict(lens=P(0x1000000), new=None, B=4, N=4, page=16, mp=8, free=P(0x2000000), F=3, tab=P(0x3000000),
             out=P(0x4000000), cu=P(0x5000000), sm=P(0x6000000), pos=P(0x7000000), tk=P(0x8000000), ws=WS, wsb=256)
    a.update(kw)
    return lib.dsa_paged_slots(a["lens"], a["new"], a["B"], a["N"], a["page"], a["mp"], a["free"], a["F"], a["tab"],
                               a["out"], a["cu"], a["sm"], a["pos"], a["tk"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(B=8193), dict(N=-1), dict(page=0), dict(mp=-1), dict(F=-1),
                                 dict(lens=None), dict(tab=None), dict(out=None), dict(cu=None), dict(sm=None),
                                 dict(pos=None), dict(tk=None), dict(free=None), dict(out=P(0x1000000)),
                                 dict(out=P(0x1000000 + 12)), dict(pos=P(0x6000000)), dict(sm=P(0x3000000 + 4)),
                                 dict(cu=P(0x2000000 + 8))])
def test_slots_refuse(lib, bad):
    assert slots(lib, **bad) == 3
    assert lib.dsa_last_error_message().decode().startswith("dsa_paged_slots")


def test_slots_refuse_a_bad_workspace(lib):
    assert slots(lib, ws=None) == 4 and slots(lib, ws=P(0x100010)) == 4 and slots(lib, wsb=255) == 4


def fwd(lib, **kw):
    a = dict(x=FAKE, xt=576, xh=0, T=4, H=1, D=576, norm=1, n=512, w=FAKE, b=None, eps=1e-6, r0=512, R=64, inter=1,
             pos=FAKE, f=FAKE, sc=1.0, out=P(0x20000), ot=576, oh=0, rows=None, nr=0, ws=WS, wsb=256)
    a.update(kw)
    return lib.dsa_norm_rope_fwd(a["x"], a["xt"], a["xh"], a["T"], a["H"], a["D"], a["norm"], a["n"], a["w"], a["b"],
                                 a["eps"], a["r0"], a["R"], a["inter"], a["pos"], a["f"], a["sc"], a["out"], a["ot"],
                                 a["oh"], a["rows"], a["nr"], a["ws"], a["wsb"], None)


BAD_ROWS = [dict(T=-1), dict(H=0), dict(D=0), dict(D=1025), dict(norm=3), dict(norm=-1), dict(n=0), dict(n=577),
            dict(norm=0, w=None), dict(norm=0, n=0), dict(eps=-1.0), dict(eps=float("nan")), dict(R=63), dict(R=-2),
            dict(r0=-1), dict(r0=513), dict(inter=2), dict(pos=None), dict(f=None), dict(sc=float("inf")),
            dict(x=None), dict(x=P(0x10001)), dict(xt=-1), dict(xh=-8)]


@pytest.mark.parametrize("bad", BAD_ROWS + [dict(b=FAKE), dict(out=None), dict(ot=575), dict(H=2, oh=64),
                                            dict(H=2, oh=576, ot=600), dict(H=2, oh=2000, ot=576), dict(rows=FAKE, nr=-1),
                                            dict(rows=FAKE, nr=1 << 31)])
def test_forward_refuses(lib, bad):
    assert fwd(lib, **bad) == 3
    assert lib.dsa_last_error_message().decode().startswith("dsa_norm_rope_fwd")


def bwd(lib, **kw):
    a = dict(g=FAKE, gt=576, gh=0, x=FAKE, xt=576, xh=0, T=4, H=1, D=576, norm=1, n=512, w=FAKE, eps=1e-6, r0=512, R=64,
             inter=1, pos=FAKE, f=FAKE, sc=1.0, dx=P(0x20000), dt=576, dh=0, dw=FAKE, db=None, acc=0, ws=WS, wsb=1 << 30)
    a.update(kw)
    return lib.dsa_norm_rope_bwd(a["g"], a["gt"], a["gh"], a["x"], a["xt"], a["xh"], a["T"], a["H"], a["D"], a["norm"],
                                 a["n"], a["w"], a["eps"], a["r0"], a["R"], a["inter"], a["pos"], a["f"], a["sc"],
                                 a["dx"], a["dt"], a["dh"], a["dw"], a["db"], a["acc"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", BAD_ROWS + [dict(g=None), dict(gt=-1), dict(dx=None), dict(dt=575), dict(db=FAKE),
                                            dict(norm=0, n=0, w=None, dw=FAKE), dict(acc=2)])
def test_backward_refuses(lib, bad):
    assert bwd(lib, **bad) == 3
    assert lib.dsa_last_error_message().decode().startswith("dsa_norm_rope_bwd")


def test_backward_workspace(lib):
    need = lib.dsa_norm_rope_bwd_workspace_size(512)
    assert need > lib.dsa_norm_rope_bwd_workspace_size(64) > lib.dsa_norm_rope_bwd_workspace_size(0) == 256
    assert bwd(lib, wsb=need - 1) == 4 and bwd(lib, ws=None) == 4


def mla(lib, **kw):
    a = dict(q=FAKE, c=FAKE, tab=FAKE, ln=FAKE, cu=None, idx=None, il=None, N=4, B=4, H=16, D=576, Dv=512, K=0, pages=8,
             page=64, mp=4, scale=0.1, sink=None, out=FAKE, lse=FAKE, ws=WS, wsb=1 << 30)
    a.update(kw)
    return lib.dsa_paged_mla(a["q"], a["c"], a["tab"], a["ln"], a["cu"], a["idx"], a["il"], a["N"], a["B"], a["H"], a["D"],
                             a["Dv"], a["K"], a["pages"], a["page"], a["mp"], a["scale"], a["sink"], a["out"], a["lse"],
                             a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [dict(N=-1), dict(B=-1), dict(H=0), dict(K=-1), dict(pages=-1), dict(page=0), dict(mp=-1),
                                 dict(D=500), dict(Dv=256), dict(N=3), dict(scale=0.0), dict(scale=float("nan")),
                                 dict(idx=FAKE), dict(K=4), dict(il=FAKE), dict(q=None), dict(out=None), dict(lse=None),
                                 dict(ln=None), dict(tab=None), dict(c=None), dict(q=P(0x10008)), dict(out=P(0x10008)),
                                 dict(c=P(0x10002)), dict(N=1 << 28, H=64, cu=FAKE)])
def test_paged_mla_refuses(lib, bad):
    assert mla(lib, **bad) == 3
    assert lib.dsa_last_error_message().decode().startswith("dsa_paged_mla")


def test_paged_mla_refuses_a_bad_workspace(lib):
    need = lib.dsa_paged_mla_workspace_size()
    assert mla(lib, ws=None) == 4 and mla(lib, ws=P(0x100010)) == 4 and mla(lib, wsb=need - 1) == 4


def topk(lib, **kw):
    a = dict(q=FAKE, c=FAKE, w=FAKE, tab=FAKE, ln=FAKE, cu=None, N=4, B=4, Hi=64, Di=128, K=64, pages=8, page=64, mp=4,
             most=256, idx=FAKE, il=None, ws=WS, wsb=1 << 30)
    a.update(kw)
    return lib.dsa_paged_indexer_topk(a["q"], a["c"], a["w"], a["tab"], a["ln"], a["cu"], a["N"], a["B"], a["Hi"], a["Di"],
                                      a["K"], a["pages"], a["page"], a["mp"], a["most"], a["idx"], a["il"], a["ws"],
                                      a["wsb"], None)


@pytest.mark.parametrize("bad", [dict(N=-1), dict(B=-1), dict(Hi=0), dict(Hi=65), dict(Di=64), dict(K=0), dict(K=2049),
                                 dict(pages=-1), dict(page=0), dict(mp=-1), dict(most=-1), dict(N=3), dict(q=None),
                                 dict(w=None), dict(idx=None), dict(ln=None), dict(tab=None), dict(c=None),
                                 dict(q=P(0x10008)), dict(c=P(0x10002)), dict(N=1 << 29, cu=FAKE)])
def test_paged_indexer_refuses(lib, bad):
    assert topk(lib, **bad) == 3
    assert lib.dsa_last_error_message().decode().startswith("dsa_paged_indexer_topk")


def test_paged_indexer_refuses_a_bad_workspace(lib):
    need = lib.dsa_paged_indexer_topk_workspace_size(4, 255)
    assert need >= 256 + 4 * 256 * 4
    assert topk(lib, ws=None) == 4 and topk(lib, ws=P(0x100010)) == 4 and topk(lib, wsb=need - 1) == 4


def test_sizes_past_what_a_kernel_counts_are_refused(lib):
    # rows are counted up to a run past the last one, positions up to a round past a row's end
    for f in (fwd, bwd):
        assert f(lib, T=2 ** 31 - 64) == 3 and f(lib, T=2 ** 30, H=2, D=64, n=64, r0=0, xt=128, xh=64, ot=128, oh=64, dt=128, dh=64,
                                                 gt=128, gh=64) == 3
        assert "T * H" in lib.dsa_last_error_message().decode()
    assert topk(lib, most=2 ** 30 + 1) == 3 and "max_len" in lib.dsa_last_error_message().decode()


def test_the_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_norm_rope_fwd(x)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_norm_rope_bwd(x)
    with pytest.raises(TypeError):
        dsa.dsa_norm_rope_fwd(x.float())
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_paged_slots(i, i.view(4, 1), i, 16)
    with pytest.raises(TypeError):
        dsa.dsa_paged_slots(i.long(), i.view(4, 1), i, 16)


def frequencies(R, base, factor, ctx, fast, slow):
    """The published rule by parts, written from its definition: wavelength against context."""
    f = base ** (-np.arange(0, R, 2) / R)
    if factor == 1:
        return f, 1.0
    dim = lambda r: R * np.log(ctx / (2 * np.pi * r)) / (2 * np.log(base))  # noqa: E731
    lo, hi = max(np.floor(dim(fast)), 0), min(np.ceil(dim(slow)), R - 1)
    keep = 1 - np.clip((np.arange(R // 2) - lo) / (hi - lo if hi > lo else 1e-3), 0, 1)
    return f / factor * (1 - keep) + f * keep, 0.1 * np.log(factor) + 1


@pytest.mark.parametrize("R,base,factor,ctx", [(64, 10000.0, 1.0, 4096), (64, 10000.0, 40.0, 4096), (128, 1e6, 4.0, 32768),
                                               (2, 500.0, 2.0, 10), (64, 10000.0, 8.0, 1)])
def test_frequencies(lib, R, base, factor, ctx):
    f, s = dsa.dsa_rope_frequencies(R, base, factor, ctx, device="cpu")
    want, scale = frequencies(R, base, factor, ctx, 32.0, 1.0)
    assert f.shape == (R // 2,) and np.all(np.abs(f.double().numpy() - want) <= 2.0 ** -24 * want * 1.0001)
    assert abs(s - scale) <= 2.0 ** -24 * scale


def test_frequencies_refuse(lib):
    for bad in (dict(rope_dim=3), dict(rope_dim=0), dict(base=1.0), dict(base=float("nan")), dict(factor=0.5),
                dict(factor=2.0, original_context=0), dict(factor=2.0, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_rope_frequencies(**{**dict(rope_dim=64, device="cpu"), **bad})


@pytest.mark.parametrize("kind,n,r0,inter", [("rms", 12, 10, True), ("layer", 16, 0, False), ("none", 0, 4, True)])
def test_the_reference_gradient_against_differences(kind, n, r0, inter):
    r = np.random.RandomState(3)
    x, g, pos, f = r.randn(3, 2, 16), r.randn(3, 2, 16), np.array([0.0, 5.0, -70.0]), np.array([1.0, 0.2, 0.03])
    w, b = (1 + 0.3 * r.randn(n), 0.3 * r.randn(n)) if n else (None, None)
    loss = lambda x, w, b: float((g * ref.norm_rope_fwd(x, kind, n, w, b, 1e-3, pos, f, r0, inter, 1.3)).sum())  # noqa: E731
    dx, dw, db, *_ = ref.norm_rope_bwd(g, x, kind, n, w, 1e-3, pos, f, r0, inter, 1.3)
    for a, d in ((x, dx),) + (((w, dw),) if n else ()) + (((b, db),) if kind == "layer" else ()):
        for at in np.ndindex(a.shape):
            old = a[at]
            a[at] = old + 1e-5
            up = loss(x, w, b)
            a[at] = old - 1e-5
            down = loss(x, w, b)
            a[at] = old
            assert abs((up - down) / 2e-5 - d[at]) < 1e-7 * max(1.0, abs(d[at])) + 1e-7
