"""Rows of a quantised cache: written by the kernel byte for byte as the format says, and read back exactly."""
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _quant_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def rows_of_every_kind(T, D, Q, g):
    """Rows of the sizes that meet the scales' borders, with channels between two codes among them."""
    x = torch.randn(T, D, generator=g)
    kind = torch.arange(T) % 9
    x[kind == 1] = (x[kind == 1] * 16).round() / 8            # few bits: ties between codes
    x[kind == 2] *= torch.exp(3 * torch.randn(D, generator=g))  # blocks of very different size
    x[kind == 3] *= 2.0 ** -60                                # below the smallest scale
    x[kind == 4] *= 2.0 ** 46                                 # near the largest one
    x[kind == 5] = 0
    x[kind == 6] = x[kind == 6].sign() * 2.0 ** torch.randint(-30, 30, (int((kind == 6).sum()), D), generator=g)
    x = x.bfloat16()
    for t in range(T):  # a largest magnitude at the border of s, one step to either side of it
        if t % 9 == 7:
            edge = torch.tensor([448.0, 2688.0, 6.0, 1.75][t // 9 % 4] * 2.0 ** (t % 5), dtype=torch.bfloat16)
            x[t, :Q].clamp_(-1, 1)
            x[t, t % Q] = (edge.view(torch.int16) + (t // 36) % 3 - 1).view(torch.bfloat16)
        if t % 9 == 8:
            x[t, (7 * t) % Q] = [float("nan"), float("inf"), -float("inf"), 2.0 ** 70, 2.0 ** 56][t // 9 % 5]
    return x


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,Q,T", [(576, 512, 83), (512, 512, 9), (128, 128, 131), (72, 64, 37), (192, 128, 1), (1024, 960, 20),
                                   (264, 256, 65), (1024, 1024, 18)])
def test_rows_are_written_as_the_format_says_and_read_back(bits, D, Q, T):
    g = torch.Generator().manual_seed(bits * 1000 + D + T)
    x = rows_of_every_kind(T, D, Q, g)
    want = ref.encode(x, Q, bits)
    n = T + 30
    slots = torch.randperm(n, generator=g)[:T].to(I32)
    slots[3::17] = -1
    keep = slots >= 0
    cache = torch.randint(0, 256, (n, want.shape[1]), generator=g, dtype=torch.uint8)
    full = cache.clone()
    full[slots[keep].long()] = want[keep]
    c = cache.to(DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    assert dsa.dsa_paged_quantize(x.to(DEV), c, bits, Q, slots.to(DEV), workspace=ws) is c
    assert torch.equal(c.cpu(), full)
    # read back by slots, among rows that are left as they are
    named = slots[keep].to(DEV)
    k = len(named)
    out = torch.full((k + 5, D + 3), 7.0, dtype=torch.bfloat16, device=DEV)
    dsa.dsa_paged_dequantize(c, named[None], torch.tensor([2, 2 + k], dtype=I32, device=DEV), bits, D, Q,
                             out=out[:, :D], workspace=ws)
    got = out.cpu()
    assert bool((got[:2] == 7).all()) and bool((got[2 + k:] == 7).all()) and bool((got[:, D:] == 7).all())
    exact = ref.decode(want[keep], D, Q, bits)
    assert torch.equal(torch.nan_to_num(got[2:2 + k, :D].double(), 99.0), torch.nan_to_num(exact, 99.0))
    assert dsa.dsa_read_device_status(ws) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_every_magnitude_of_bf16(bits):
    """Each positive bf16 against each of a few largest magnitudes of its row."""
    mags = torch.arange(0, 0x7f80, 1, dtype=torch.int16)[::7].view(torch.bfloat16)
    rows = []
    for top in (1.0, 1.3125, 1.328125, 1.75, 1.7578125, 5.0):
        v = mags[mags.float() <= top * 2.0 ** 20]
        v = v[-(len(v) // 63 * 63):].reshape(-1, 63)
        rows.append(torch.cat([torch.full((len(v), 1), top * 2.0 ** 20).bfloat16(), v], 1))
    x = torch.cat(rows)
    x = torch.cat([x, -x[:, [0]] * 0, x[:, :7]], 1)[:, :72].contiguous()
    c = torch.zeros(len(x), dsa.paged_quant_row_bytes(72, bits, 64), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(x.to(DEV), c, bits, 64)
    assert torch.equal(c.cpu(), ref.encode(x, 64, bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("stride,shift", [(600, 8), (577, 0), (584, 3), (0, 0)])
def test_strides_of_the_input(bits, stride, shift):
    g = torch.Generator().manual_seed(stride)
    T = 21
    flat = torch.randn(T * 600 + 16, generator=g).bfloat16()
    x = flat.as_strided((T, 576), (stride, 1), shift)
    c = torch.zeros(T, 1, dsa.paged_quant_row_bytes(576, bits), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(flat.to(DEV).as_strided((T, 576), (stride, 1), shift), c, bits)
    assert torch.equal(c.cpu()[:, 0], ref.encode(x.contiguous(), 512, bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("page,lens,first", [(16, [1, 0, 33, 16, 200], [0, 5, 15, 16, 1]), (1, [3, 70], None),
                                             (48, [0, 0, 100], None), (64, [500], [3]), (7, [40] * 30, [1] * 30)])
def test_requests_are_read_back_through_their_tables(bits, page, lens, first):
    g = torch.Generator().manual_seed(page)
    start = first or [0] * len(lens)
    need = [-(-(n + s) // page) for n, s in zip(lens, start)]
    pages = sum(need) + 2
    x = torch.randn(pages * page, 576, generator=g).bfloat16()
    cache = torch.zeros(pages, page, dsa.paged_quant_row_bytes(576, bits), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(x.to(DEV), cache, bits)
    perm = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(need)), -5, dtype=I32)
    for b, k in enumerate(need):
        table[b, :k] = torch.tensor([perm.pop() for _ in range(k)], dtype=I32)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    d = lambda v: torch.tensor(v, dtype=I32, device=DEV)  # noqa: E731
    out = dsa.dsa_paged_dequantize(cache, table.to(DEV), d(cu), bits, 576, first=None if first is None else d(first),
                                   N=cu[-1], workspace=ws)
    flat = cache.cpu().view(pages * page, -1)
    at = [int(table[b, p // page]) * page + p % page for b, n in enumerate(lens) for p in range(start[b], start[b] + n)]
    assert torch.equal(out.cpu().double(), ref.decode(flat[at], 576, 512, bits))
    assert dsa.dsa_read_device_status(ws) == 0


def test_bad_rows_and_pages_are_reported():
    x = torch.randn(4, 128, device=DEV).bfloat16()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    c = torch.zeros(6, 144, dtype=torch.uint8, device=DEV)
    d = lambda v: torch.tensor(v, dtype=I32, device=DEV)  # noqa: E731
    dsa.dsa_paged_quantize(x, c, 8, out_rows=d([0, 6, -2, 5]), workspace=ws)
    assert dsa.dsa_read_device_status(ws) == 6 and dsa.dsa_read_device_status(ws) == 0
    assert bool((c[1:5] == 0).all()) and bool((c[[0, 5]] != 0).any(1).all())
    # pages 9 and -1, a position beyond the table and one before its start
    pages = c.view(3, 2, 144)
    for table, first, bad in (([[0, 9, 2]], [0], [2, 3]), ([[0, -1, 2]], [0], [2, 3]), ([[0, 1, 2]], [1], [5]),
                              ([[0, 1, 2]], [-1], [0])):
        out = dsa.dsa_paged_dequantize(pages, d(table), d([0, 6]), 8, 128, first=d(first), N=6, workspace=ws)
        assert dsa.dsa_read_device_status(ws) == 6
        assert bool((out[bad] == 0).all())
    dsa.dsa_paged_dequantize(pages, d([[0, 1, 2]]), d([0, 6]), 8, 128, N=6, workspace=ws)
    assert dsa.dsa_read_device_status(ws) == 0


def test_calls_of_nothing():
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    c = torch.zeros(0, 16, 656, dtype=torch.uint8, device=DEV)
    none = torch.zeros(0, 576, dtype=torch.bfloat16, device=DEV)
    i = torch.zeros(0, dtype=I32, device=DEV)
    dsa.dsa_paged_quantize(none, c, 8, out_rows=i, workspace=ws)
    assert dsa.dsa_paged_dequantize(c, i.view(0, 3), torch.zeros(1, dtype=I32, device=DEV), 8, 576, N=0, workspace=ws).shape == (0, 576)
    one = dsa.dsa_paged_quantize(torch.ones(1, 576, dtype=torch.bfloat16, device=DEV), c, 8,
                                 out_rows=torch.full((1,), -1, dtype=I32, device=DEV), workspace=ws)
    assert one is c and dsa.dsa_read_device_status(ws) == 0


def test_the_binding_refuses_other_shapes():
    x = torch.zeros(4, 576, dtype=torch.bfloat16, device=DEV)
    c = torch.zeros(4, 1, 656, dtype=torch.uint8, device=DEV)
    cu = torch.tensor([0, 4], dtype=I32, device=DEV)
    tab = torch.zeros(1, 4, dtype=I32, device=DEV)
    for bad in (lambda: dsa.dsa_paged_quantize(x, c, 4), lambda: dsa.dsa_paged_quantize(x[:, None], c, 8),
                lambda: dsa.dsa_paged_quantize(x.t(), c, 8), lambda: dsa.dsa_paged_quantize(x, c, 8, out_rows=cu),
                lambda: dsa.dsa_paged_dequantize(c, tab, cu, 8, 576), lambda: dsa.dsa_paged_dequantize(c, tab, cu, 4, 576, N=4),
                lambda: dsa.dsa_paged_dequantize(c, tab, cu, 8, 576, N=4, out=x[:3]),
                lambda: dsa.dsa_paged_dequantize(c, tab.view(4, 1), cu, 8, 576, N=4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dsa.DsaError):
        dsa.dsa_paged_quantize(x, c[:3], 8)


@pytest.mark.parametrize("bits", [8, 4])
def test_many_rows_of_many_requests_are_read_back(bits):
    # enough rows for the wider blocks, requests of none in between, and rows of out that are no request's
    D, Q, page = 72, 64, 16
    g = torch.Generator().manual_seed(bits)
    lens = torch.randint(0, 290, (420,), generator=g)
    lens[torch.rand(420, generator=g) < 0.2] = 0
    lens[100:140] = 0
    need = (lens + page - 1) // page
    pages = int(need.sum())
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((420, int(need.max())), -1, dtype=torch.int32)
    at = 0
    for b in range(420):
        table[b, :need[b]] = perm[at:at + int(need[b])]
        at += int(need[b])
    cache = torch.zeros(pages, page, dsa.paged_quant_row_bytes(D, bits, Q), dtype=torch.uint8, device=DEV)
    x = torch.randn(pages * page, D, generator=g).bfloat16().to(DEV)
    dsa.dsa_paged_quantize(x, cache, bits, quant_dim=Q)
    cu = torch.zeros(421, dtype=torch.int32)
    cu[1:] = lens.cumsum(0)
    cu += 7
    N = int(cu[-1]) + 9
    assert N > 64 * 4 * 152
    out = torch.full((N, D), 5.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_dequantize(cache, table.to(DEV), cu.to(DEV), bits, D, quant_dim=Q, out=out, workspace=ws)
    assert dsa.dsa_read_device_status(ws) == 0
    rows = torch.cat([table[b, torch.arange(int(lens[b])) // page].long() * page + torch.arange(int(lens[b])) % page
                      for b in range(420)])
    want = ref.decode(cache.view(-1, cache.shape[2])[rows.to(DEV)], D, Q, bits)
    got = out.cpu().double()
    assert bool((got[:7] == 5).all()) and bool((got[N - 9:] == 5).all())
    assert torch.equal(got[7:N - 9], want)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,Q", [(576, 512), (72, 64)])
@pytest.mark.parametrize("stride,shift", [(0, 0), (16, 16), (8, 0), (16, 8), (1, 0), (3, 5)])
def test_strides_of_the_output(bits, D, Q, stride, shift):
    # rows that begin at multiples of 32, 16 and 2 bytes; what lies between them is left as it was
    g = torch.Generator().manual_seed(D + stride)
    cache = torch.zeros(70, 1, dsa.paged_quant_row_bytes(D, bits, Q), dtype=torch.uint8, device=DEV)
    dsa.dsa_paged_quantize(torch.randn(70, D, generator=g).bfloat16().to(DEV), cache, bits, quant_dim=Q)
    rows = torch.randperm(70, generator=g).to(I32)
    flat = torch.full((70 * (D + stride) + shift,), 9.0, dtype=torch.bfloat16, device=DEV)
    out = flat[shift:].view(70, D + stride)[:, :D]
    cu = torch.tensor([0, 70], dtype=I32, device=DEV)
    dsa.dsa_paged_dequantize(cache, rows[None].to(DEV), cu, bits, D, quant_dim=Q, out=out)
    want = ref.decode(cache.view(70, -1).cpu()[rows.long()], D, Q, bits)
    assert torch.equal(out.cpu().double(), want)
    rest = flat[shift:].view(70, D + stride)[:, D:]
    assert bool((rest == 9).all()) and bool((flat[:shift] == 9).all())
