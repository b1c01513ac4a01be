"""CPU checks of the calls over a quantised cache: what the library and the binding refuse before anything is launched,
and the tests' own form of a row."""
import ctypes
import inspect

import pytest
import torch

import sparse_attention_mla_gb300 as dsa
from sparse_attention_mla_gb300 import build_ext

import _quant_ref as ref

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: validation fails before any device use
WS = P(0x100000)


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return dsa.load_library()


def test_names(lib):
    for name in ("dsa_paged_quantize", "dsa_paged_dequantize", "dsa_paged_mla_quant"):
        assert callable(getattr(dsa, name)) and name in dsa.declared_symbols() and hasattr(lib, name)
        doc = getattr(dsa, name).__doc__
        assert "dsa_read_device_status" in doc and "paged_workspace_size" in doc and "dropped" in doc


@pytest.mark.parametrize("D,Q", [(576, 512), (512, 512), (128, 128), (192, 128), (72, 64), (1024, 1024), (1024, 960)])
@pytest.mark.parametrize("bits", [8, 4])
def test_row_bytes(lib, D, Q, bits):
    n = dsa.paged_quant_row_bytes(D, bits, Q)
    assert n == ref.layout(D, Q, bits)[3] and n % 16 == 0 and n >= Q * bits // 8 + 4 + 2 * (D - Q)


@pytest.mark.parametrize("D,Q,bits", [(576, 512, 5), (576, 500, 8), (576, 0, 8), (580, 512, 4), (500, 512, 4),
                                      (1088, 1024, 8), (512, -64, 4), (96, 96, 4)])
def test_no_such_rows(lib, D, Q, bits):
    assert lib.dsa_paged_quant_row_bytes(D, Q, bits) == 0
    with pytest.raises(ValueError, match="no such rows"):
        dsa.paged_quant_row_bytes(D, bits, Q)
    assert quantize(lib, D=D, Q=Q, bits=bits) == 3 and dequantize(lib, D=D, Q=Q, bits=bits, ot=2048) == 3


def quantize(lib, **kw):
    a = dict(x=FAKE, xt=576, T=4, D=576, Q=512, bits=8, c=P(0x1000000), n=64, rows=FAKE, ws=WS, wsb=256)
    a.update(kw)
    return lib.dsa_paged_quantize(a["x"], a["xt"], a["T"], a["D"], a["Q"], a["bits"], a["c"], a["n"], a["rows"], a["ws"],
                                  a["wsb"], None)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(xt=-1), dict(n=-1), dict(n=2 ** 31), dict(n=3, rows=None), dict(x=None),
                                 dict(c=None), dict(x=P(0x10001)), dict(c=P(0x1000008)), dict(x=P(0x1000000 + 64 * 656 - 2)),
                                 dict(x=P(0x1000000 - 4 * 1152 + 2))])
def test_quantize_refuses(lib, bad):
    assert quantize(lib, **bad) == 3
    assert lib.dsa_last_error_message().decode().startswith("dsa_paged_quantize")


def dequantize(lib, **kw):
    a = dict(c=P(0x1000000), tab=FAKE, first=None, cu=FAKE, N=4, B=2, D=576, Q=512, bits=4, pages=8, page=16, mp=4,
             out=P(0x20000), ot=576, ws=WS, wsb=256)
    a.update(kw)
    return lib.dsa_paged_dequantize(a["c"], a["tab"], a["first"], a["cu"], a["N"], a["B"], a["D"], a["Q"], a["bits"],
                                    a["pages"], a["page"], a["mp"], a["out"], a["ot"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [dict(N=-1), dict(B=-1), dict(pages=-1), dict(page=0), dict(mp=-1), dict(ot=575),
                                 dict(out=None), dict(cu=None), dict(tab=None), dict(c=None), dict(out=P(0x20001)),
                                 dict(c=P(0x1000004)), dict(out=P(0x1000000 + 128 * 432 - 2)), dict(ot=-576)])
def test_dequantize_refuses(lib, bad):
    assert dequantize(lib, **bad) == 3
    assert lib.dsa_last_error_message().decode().startswith("dsa_paged_dequantize")


def mla(lib, **kw):
    a = dict(q=FAKE, c=FAKE, tab=FAKE, ln=FAKE, cu=None, idx=None, il=None, N=4, B=4, H=16, D=576, Dv=512, bits=4, K=0,
             pages=8, page=64, mp=4, scale=0.1, sink=None, out=FAKE, lse=FAKE, ws=WS, wsb=1 << 30)
    a.update(kw)
    return lib.dsa_paged_mla_quant(a["q"], a["c"], a["tab"], a["ln"], a["cu"], a["idx"], a["il"], a["N"], a["B"], a["H"],
                                   a["D"], a["Dv"], a["bits"], a["K"], a["pages"], a["page"], a["mp"], a["scale"],
                                   a["sink"], a["out"], a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [dict(N=-1), dict(B=-1), dict(H=0), dict(K=-1), dict(pages=-1), dict(page=0), dict(mp=-1),
                                 dict(D=500), dict(Dv=256), dict(N=3), dict(scale=0.0), dict(scale=float("nan")),
                                 dict(bits=6), dict(bits=16), dict(idx=FAKE), dict(K=4), dict(il=FAKE), dict(q=None),
                                 dict(out=None), dict(lse=None), dict(ln=None), dict(tab=None), dict(c=None),
                                 dict(q=P(0x10008)), dict(out=P(0x10008)), dict(c=P(0x10002)),
                                 dict(N=1 << 28, H=64, cu=FAKE)])
def test_paged_mla_quant_refuses(lib, bad):
    assert mla(lib, **bad) == 3
    assert lib.dsa_last_error_message().decode().startswith("dsa_paged_mla_quant")


def test_bad_workspaces_are_refused(lib):
    need = lib.dsa_paged_mla_quant_workspace_size()
    assert need >= 256 and dsa.paged_workspace_size("mla_quant", 4, 64) == need
    assert dsa.paged_workspace_size("quantize") == dsa.paged_workspace_size("dequantize") == 256
    for f, n in ((quantize, 256), (dequantize, 256), (mla, need)):
        assert f(lib, ws=None) == 4 and f(lib, ws=P(0x100010)) == 4 and f(lib, wsb=n - 1) == 4


def test_the_binding_refuses():
    x = torch.zeros(4, 576, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(4, 1, 656, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_paged_quantize(x, c, 8)
    with pytest.raises(TypeError):
        dsa.dsa_paged_quantize(x.float(), c, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_paged_dequantize(c, i[None], i[:2], 8, 576, N=4)
    with pytest.raises(TypeError):
        dsa.dsa_paged_dequantize(c, i[None], i[:2].long(), 8, 576, N=4)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_paged_mla_quant(x[:, None], c, i[:, None], i, 0.1, 8)


@pytest.mark.parametrize("bits", [8, 4])
def test_the_reference_rows(bits):
    """Values that a row can hold come back as they were, others are off by half a step at most."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(6, 72, generator=g).bfloat16()
    x[1] = 0
    x[2, :64] *= 2.0 ** -30
    x[3, 7] = float("inf")
    x[4, 0] = 2.0 ** 70
    rows = ref.encode(x, 64, bits)
    y = ref.decode(rows, 72, 64, bits)
    assert torch.equal(y[:, 64:], x[:, 64:].double()) and bool(torch.isnan(y[3:5, :64]).all()) and bool((y[1, :64] == 0).all())
    keep = [0, 1, 2, 5]
    again = ref.decode(ref.encode(y[keep].bfloat16(), 64, bits), 72, 64, bits)
    v, w = x[keep, :64].double(), y[keep, :64]
    if bits == 8:  # (the smallest step is 2^-9 s, and s < amax / 224)
        assert torch.equal(again, y[keep])
        assert bool(((w - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -10 / 224 * v.abs().amax(1, keepdim=True)).all())
    else:  # half a step is amax / 6 of a block at most, a block's scale is off by 1/16 of itself
        top = v.reshape(-1, 4, 16).abs().amax(2).repeat_interleave(16, 1)
        assert bool(((w - v).abs() <= top / 6 * 17 / 16).all())


@pytest.mark.parametrize("name", ["dsa_paged_quantize", "dsa_paged_dequantize", "dsa_paged_mla_quant"])
def test_a_call_with_a_workspace_says_how_its_errors_are_read(name):
    call = getattr(dsa, name)
    doc = " ".join(call.__doc__.split())
    assert inspect.signature(call).parameters["workspace"].default is None
    assert all(w in doc for w in ("dsa_read_device_status", "paged_workspace_size", "zeroed once", "dropped"))
