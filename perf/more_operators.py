"""The operators of a serving step over a quantised cache, in their plain form and through the framework.

Three operators: rows quantised as they are written to a cache of 8 or 4 bits and read back (``dsa_paged_quantize``,
``dsa_paged_dequantize``), the reading of whole contexts (``dsa_paged_dequantize``), and the attention of new tokens over
such a cache of latents (``dsa_paged_mla_quant``).

A row of D channels holds its first Q as codes and the rest as they are:
8 bits: Q codes e4m3, an fp32 scale s, 12 zero bytes, the rest in bf16; a value is code * s.
4 bits: Q / 2 bytes of codes e2m1 (the even channel in the low half), Q / 16 block scales e4m3, s, zero bytes up to a
multiple of 16, the rest; a value is code * block * s.
s is the smallest power of two in [2^-48, 2^48] with which the row's largest magnitude fits (448, or 6 * 448); a block's
scale is its largest magnitude / (6 s), rounded; codes are rounded to nearest, ties to even, at most 448 or 6."""
import math

import torch

own = False

DV = 512
DEV = "cuda"


# ----------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the latents of a decode step of 256 requests, to their slots in a cache of 8 bits
        {"name": "write, 256 latents, 8 bits", "op": "write", "T": 256, "D": 576, "Q": 512, "bits": 8, "wide": 0},
        # a chunk of a prompt, to a cache of 4 bits, from the latent part of a wider projection
        {"name": "write, 8191 latents, 4 bits", "op": "write", "T": 8191, "D": 576, "Q": 512, "bits": 4, "wide": 1536},
        # rows of 128 channels (index keys) of a whole long prompt, 8 bits
        {"name": "write, 131104 rows of 128", "op": "write", "T": 131104, "D": 128, "Q": 128, "bits": 8, "wide": 0},
        # one request's prefix in front of its next chunk
        {"name": "read, 1 x 6001, 8 bits", "op": "read", "B": 1, "L": 6001, "D": 576, "Q": 512, "bits": 8, "page": 16},
        # prefixes of several requests, very different in length
        {"name": "read, 12 x 30000, 4 bits", "op": "read", "B": 12, "L": 30000, "D": 576, "Q": 512, "bits": 4, "page": 64},
        # the smallest attention call: one request, a short context, a few local heads
        {"name": "attention, 1 x 1000, 4 bits", "op": "mla", "B": 1, "L": 1000, "H": 16, "nq": 1, "D": 576, "page": 16,
         "K": 0, "sink": False, "bits": 4},
        # a serving batch of mixed lengths, all heads on one GPU
        {"name": "attention, 64 x 16k, 4 bits", "op": "mla", "B": 64, "L": 16384, "H": 64, "nq": 1, "D": 576, "page": 64,
         "K": 0, "sink": False, "bits": 4},
        # the same over 8 bits
        {"name": "attention, 64 x 16k, 8 bits", "op": "mla", "B": 64, "L": 16384, "H": 64, "nq": 1, "D": 576, "page": 64,
         "K": 0, "sink": False, "bits": 8},
        # one long context, twice as many heads, two tokens (one drafted)
        {"name": "attention, 1 x 131k, 128 heads", "op": "mla", "B": 1, "L": 131071, "H": 128, "nq": 2, "D": 576,
         "page": 64, "K": 0, "sink": False, "bits": 4},
        # no position channels, a few local heads, many middling requests, pages of an odd size
        {"name": "attention, 96 x 4k, 8 heads", "op": "mla", "B": 96, "L": 4097, "H": 8, "nq": 1, "D": 512, "page": 48,
         "K": 0, "sink": True, "bits": 4},
        # the sparse form: every token attends to its own 2048 selected positions
        {"name": "attention, 48 x 2048 selected", "op": "mla", "B": 48, "L": 20000, "H": 64, "nq": 1, "D": 576,
         "page": 64, "K": 2048, "sink": True, "bits": 8},
        # the same for four drafted tokens of few requests, 4 bits
        {"name": "attention, 3 x 4 x 1999 selected", "op": "mla", "B": 3, "L": 50000, "H": 32, "nq": 4, "D": 576,
         "page": 64, "K": 1999, "sink": False, "bits": 4},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, bits = rng.choice(["write", "read", "mla", "mla", "mla"]), rng.choice([4, 8])
    d, q = rng.choice([(576, 512), (576, 512), (512, 512), (128, 128), (192, 128), (72, 64)])
    if op == "write":
        return {"op": op, "T": _log(rng, 1, (1 << 24) // d), "D": d, "Q": q, "bits": bits, "wide": rng.choice([0, 0, 8, 64])}
    page = rng.choice([1, 16, 48, 64, 128])
    if op == "read":
        b = _log(rng, 1, 64)
        return {"op": op, "B": b, "L": _log(rng, 1, (1 << 26) // (b * d)), "D": d, "Q": q, "bits": bits, "page": page}
    b, nq = _log(rng, 1, 128), rng.choice([1, 1, 2, 4])
    h, k = rng.choice([1, 5, 8, 16, 24, 40, 64, 128]), rng.choice([0, 0, _log(rng, 1, 2048)])
    return {"op": op, "B": b, "L": _log(rng, 1, min(131072, 524288 // b, (1 << 25) // (b * nq * h))), "H": h, "nq": nq,
            "D": rng.choice([512, 576]), "page": page, "K": k, "sink": rng.random() < 0.3, "bits": bits}


def _lens(b, most):
    """Mixed lengths from about a quarter of the longest up to it, the same for every seed."""
    f = [((i + 1) * 0.6180339887498949) % 1.0 for i in range(b)]
    return [most if i == 0 else max(1, int(most * (0.25 + 0.75 * f[i]))) for i in range(b)]


def _contexts(case):
    """Lengths of the requests, new tokens included; now and then fewer than the new tokens (rows that see nothing)."""
    nq = case.get("nq", 1)
    return [n if i % 5 == 3 else max(n, nq) for i, n in enumerate(_lens(case["B"], case["L"]))]


# --------------------------------------------------------------------------------------------- quantised rows
def _codes(x, q, bits):
    """Codes of rows x [T, D] (as the numbers that they are), block scales (None for 8 bits) and s [T, 1], in fp32."""
    v = x[:, :q].float()
    most = v.abs().amax(1, keepdim=True)
    m, e = torch.frexp(most)  # most = m 2^e, m in [1/2, 1)
    # 448 = 0.875 2^9, 6 * 448 = 0.65625 2^12
    e = e - 9 + (m > 0.875).to(e.dtype) if bits == 8 else e - 12 + (m > 0.65625).to(e.dtype)
    s = torch.ldexp(torch.ones_like(most), torch.where(most > 0, e, -48).clamp(-48, 48))
    v = v / s
    if bits == 8:
        return _rounded(v, 3, -6, 448.0), None, s
    blocks = v.reshape(v.shape[0], q // 16, 16)
    scale = _rounded(blocks.abs().amax(2) / 6.0, 3, -6, 448.0)
    v = blocks / torch.where(scale > 0, scale, torch.inf)[:, :, None]
    return _rounded(v, 1, 0, 6.0).reshape(v.shape[0], q), scale, s


def _rounded(v, bits, lowest, most):
    """To the nearest number with so many bits after the leading one, subnormal below 2^lowest; ties to even."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=lowest) - bits)
    return (torch.round(v / step) * step).clamp(-most, most)


def _values(codes, scale, s):
    if scale is not None:
        codes = (codes.reshape(*scale.shape, 16) * scale[:, :, None]).reshape(codes.shape)
    return codes * s


def _row_bytes(d, q, bits):
    return _tail_at(q, bits) + -(-2 * (d - q) // 16) * 16


def _tail_at(q, bits):
    return -(-(q + 4 if bits == 8 else q // 2 + q // 16 + 4) // 16) * 16


def _packed(x, q, bits):
    """The bytes of quantised rows, uint8 [T, row bytes]."""
    t, d = x.shape
    out = torch.zeros(t, _row_bytes(d, q, bits), dtype=torch.uint8, device=DEV)
    codes, scale, s = _codes(x, q, bits)
    at = q if bits == 8 else q // 2 + q // 16
    if bits == 8:
        out[:, :q] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        mag = codes.abs()
        n = torch.where(mag < 2, 2 * mag, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
        n = n + 8 * torch.signbit(codes).to(torch.uint8)
        out[:, : q // 2] = n[:, 0::2] + 16 * n[:, 1::2]
        out[:, q // 2 : at] = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    out[:, at : at + 4] = s.view(torch.uint8)
    tail = _tail_at(q, bits)
    out[:, tail : tail + 2 * (d - q)] = x[:, q:].contiguous().view(torch.uint8)
    return out


def _unpacked(rows, d, q, bits, dtype):
    """The values of quantised rows uint8 [T, row bytes] -> [T, D]."""
    at, tail = q if bits == 8 else q // 2 + q // 16, _tail_at(q, bits)
    s = rows[:, at : at + 4].contiguous().view(torch.float32).to(dtype)
    if bits == 8:
        v = rows[:, :q].contiguous().view(torch.float8_e4m3fn).to(dtype) * s
    else:
        n = torch.stack([rows[:, : q // 2] & 15, rows[:, : q // 2] >> 4], -1).flatten(1)
        mag = (n & 7).to(dtype)
        mag = torch.where(mag < 4, mag / 2, torch.where(mag < 6, mag - 2, 2 * mag - 8))
        scale = rows[:, q // 2 : at].contiguous().view(torch.float8_e4m3fn).to(dtype)
        v = _values(torch.where(n > 7, -mag, mag), scale, s)
    rest = rows[:, tail : tail + 2 * (d - q)].contiguous().view(torch.bfloat16).to(dtype)
    return torch.cat([v, rest], 1)


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _latents(t, d, q, g, norms=True):
    """Rows as they reach a cache: a normalised part whose channels differ in size by their weight, and position channels."""
    x = torch.randn(t, d, generator=g, device=DEV)
    if norms:
        x[:, :q] *= torch.exp(0.5 * torch.randn(q, generator=g, device=DEV))
    return x.bfloat16()


def _pages(lens, page, g, spare):
    """A table of randomly placed pages for requests of these lengths, and the number of pages."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    wide = max(1, max(need))
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device=DEV)
    counts = torch.tensor(need, device=DEV)
    table[torch.arange(wide, device=DEV)[None, :] < counts[:, None]] = perm[: sum(need)]
    return table, total


def _cache(total, page, d, q, bits, g):
    """A cache of quantised rows, all of them written."""
    out = torch.empty(total * page, _row_bytes(d, q, bits), dtype=torch.uint8, device=DEV)
    for lo in range(0, total * page, 1 << 16):
        n = min(1 << 16, total * page - lo)
        out[lo : lo + n] = _packed(_latents(n, d, q, g), q, bits)
    return out.reshape(total, page, -1)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op, d, bits = case["op"], case["D"], case["bits"]
    s["ws"] = torch.zeros(256, dtype=torch.uint8, device=DEV)
    if op == "write":
        t, q = case["T"], case["Q"]
        # rows of a wider tensor, when a projection gives more than the latent
        wide = torch.zeros(t, case["wide"] + d, dtype=torch.bfloat16, device=DEV)
        wide[:, case["wide"]:] = _latents(t, d, q, g)
        s["x"] = wide[:, case["wide"]:]
        n = t + t // 2 + 64
        s["cache"] = torch.zeros(n, 1, _row_bytes(d, q, bits), dtype=torch.uint8, device=DEV)
        s["slots"] = torch.randperm(n, generator=g, device=DEV)[:t].to(torch.int32)
        s["cu"] = _ints([0, t])
        s["out"] = torch.empty(t, d, dtype=torch.bfloat16, device=DEV)
        return s
    lens, page = _contexts(case), case["page"]
    table, total = _pages(lens, page, g, 4)
    s["table"], s["seq_lens"] = table, _ints(lens)
    if op == "read":
        s["cache"] = _cache(total, page, d, case["Q"], bits, g)
        ends = [sum(lens[: i + 1]) for i in range(len(lens))]
        s["cu"], s["N"] = _ints([0] + ends), ends[-1]
        s["out"] = torch.empty(ends[-1], d, dtype=torch.bfloat16, device=DEV)
        return s
    b, nq, h = case["B"], case["nq"], case["H"]
    s["cache"] = _cache(total, page, d, DV, bits, g)
    s["cu_q"] = _ints([i * nq for i in range(b + 1)])
    n = b * nq
    s["q"] = torch.randn(n, h, d, generator=g, device=DEV).bfloat16()
    s["scale"] = d ** -0.5
    s["sink"] = torch.randn(h, generator=g, device=DEV) if case["sink"] else None
    s["topk_idx"] = s["topk_len"] = None
    if case["K"]:
        k = case["K"]
        vis = _visible(s)
        # a random increasing choice: one position from each of k' equal pieces of the visible range
        cnt = torch.minimum(vis, torch.full_like(vis, k)).clamp(min=0)
        j = torch.arange(k, device=DEV)[None, :]
        c = cnt.clamp(min=1)[:, None]
        lo, hi = j * vis[:, None] // c, (j + 1) * vis[:, None] // c
        u = torch.rand(n, k, generator=g, device=DEV, dtype=torch.float64)
        idx = lo + torch.floor(u * (hi - lo)).long()
        s["topk_idx"] = torch.where(j < cnt[:, None], idx, -1).to(torch.int32)
        s["topk_len"] = cnt.to(torch.int32)
    s["out"] = torch.empty(n, h, DV, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(n, h, dtype=torch.float32, device=DEV)
    if own:
        import sparse_attention_mla_gb300 as dsa

        s["ws"] = torch.zeros(dsa.paged_workspace_size("mla_quant"), dtype=torch.uint8, device=DEV)
    return s


def _visible(s):
    """Positions that each query token sees (its own included)."""
    nq = s["nq"]
    j = torch.arange(nq, device=DEV)
    return (s["seq_lens"].long()[:, None] - nq + j[None, :] + 1).clamp(min=0).reshape(-1)


# ------------------------------------------------------------------------------------------------- plain forms
def _row_numbers(s, pos):
    """Cache rows [B, S] of positions [B, S] (in range)."""
    page = s["page"]
    return torch.gather(s["table"].long(), 1, pos // page) * page + pos % page


def _every_position(s):
    """The cache rows of all positions up to the longest request's end [B, S] (past a request's end its last one)."""
    most = int(s["table"].shape[1]) * s["page"]
    pos = torch.arange(most, device=DEV)[None, :].expand(s["B"], most)
    return _row_numbers(s, torch.minimum(pos, (s["seq_lens"].long() - 1)[:, None]))


def _write_plain(s):
    x, q, bits = s["x"], s["Q"], s["bits"]
    rows = s["cache"].reshape(-1, s["cache"].shape[2])
    at = s["slots"].long()
    rows[at] = _packed(x, q, bits)
    return _unpacked(rows[at], s["D"], q, bits, torch.float32).bfloat16()


def _read_plain(s):
    rows = s["cache"].reshape(-1, s["cache"].shape[2])
    t = torch.arange(s["N"], device=DEV)
    r = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    pos = t - s["cu"].long()[r]
    at = s["table"].long()[r, pos // s["page"]] * s["page"] + pos % s["page"]
    return _unpacked(rows[at], s["D"], s["Q"], s["bits"], torch.float32).bfloat16()


def _mla_plain(s):
    b, nq, h, d, k = s["B"], s["nq"], s["H"], s["D"], s["K"]
    rows = s["cache"].reshape(-1, s["cache"].shape[2])
    q = s["q"].float().reshape(b, nq * h, d) * s["scale"]
    if k:
        idx = s["topk_idx"].long().reshape(b, nq * k)
        kv = _unpacked(rows[_row_numbers(s, idx.clamp(min=0)).reshape(-1)], d, DV, s["bits"], torch.float32)
        kv = kv.reshape(b * nq, k, d)
        z = torch.matmul(q.reshape(b * nq, h, d), kv.transpose(1, 2))
        seen = (s["topk_idx"] >= 0)[:, None, :]
    else:
        at = _every_position(s)
        most = at.shape[1]
        kv = _unpacked(rows[at.reshape(-1)], d, DV, s["bits"], torch.float32).reshape(b, most, d)
        z = torch.matmul(q, kv.transpose(1, 2)).reshape(b * nq, h, most)
        seen = (torch.arange(most, device=DEV)[None, :] < _visible(s)[:, None])[:, None, :]
    z = torch.where(seen, z, -torch.inf)
    top = z.amax(-1, keepdim=True)
    if s["sink"] is not None:
        top = torch.maximum(top, s["sink"][None, :, None])
    top = torch.where(top == -torch.inf, 0.0, top)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"][None, :, None] - top)
    lse = (top + torch.log(total))[..., 0]
    p = p / torch.where(total > 0, total, 1.0)
    if k:
        out = torch.matmul(p, kv[..., :DV])
    else:
        out = torch.matmul(p.reshape(b, nq * h, -1), kv[..., :DV]).reshape(b * nq, h, DV)
    return out.bfloat16(), lse


# ------------------------------------------------------------------------------------------------------- a pass
def run(s):
    op = s["op"]
    if not own:
        if op == "write":
            return _write_plain(s)
        return _read_plain(s) if op == "read" else _mla_plain(s)
    import sparse_attention_mla_gb300 as dsa

    if op == "write":
        # the rows that were written, read back by their slots (pages of one row)
        dsa.dsa_paged_quantize(s["x"], s["cache"], s["bits"], quant_dim=s["Q"], out_rows=s["slots"], workspace=s["ws"])
        return dsa.dsa_paged_dequantize(s["cache"], s["slots"][None, :], s["cu"], s["bits"], s["D"], quant_dim=s["Q"],
                                        out=s["out"], workspace=s["ws"])
    if op == "read":
        return dsa.dsa_paged_dequantize(s["cache"], s["table"], s["cu"], s["bits"], s["D"], quant_dim=s["Q"],
                                        out=s["out"], workspace=s["ws"])
    return dsa.dsa_paged_mla_quant(s["q"], s["cache"], s["table"], s["seq_lens"], s["scale"], s["bits"], cu_q=s["cu_q"],
                                   topk_idx=s["topk_idx"], topk_len=s["topk_len"], attn_sink=s["sink"], out=s["out"],
                                   lse=s["lse"], workspace=s["ws"])


def _stored(d, q, bits):
    """Bytes of a row that mean something."""
    return (q + 4 if bits == 8 else q // 2 + q // 16 + 4) + 2 * (d - q)


def work(case):
    op, d, bits = case["op"], case["D"], case["bits"]
    if op == "write":  # read, written, read back, written out
        t = case["T"]
        return {"bytes": t * (4 * d + 2 * _stored(d, case["Q"], bits) + 8), "flops": 6 * t * d}
    lens = _contexts(case)
    if op == "read":
        return {"bytes": sum(lens) * (2 * d + _stored(d, case["Q"], bits)), "flops": 2 * sum(lens) * d}
    b, nq, h, k = case["B"], case["nq"], case["H"], case["K"]
    vis = [max(0, n - nq + j + 1) for n in lens for j in range(nq)]
    pairs = sum(min(v, k) for v in vis) if k else sum(vis)
    rows = min(pairs, sum(lens)) if k else sum(lens)
    moved = rows * _stored(d, DV, bits) + b * nq * h * (2 * d + 2 * DV + 4) + 4 * b * nq * k
    return {"bytes": moved, "flops": 2 * h * (d + DV) * pairs}


# ------------------------------------------------------------------------------- 64 bits, from the definitions
def _tables64():
    """The magnitudes of e2m1 and of e4m3 by code."""
    e2m1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    e4m3 = [(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)]
    return [torch.tensor(t, dtype=torch.float64, device=DEV) for t in (e2m1, e4m3)]


def _nearest(v, table):
    """Codes of the nearest magnitudes in the table, ties to the even code."""
    hi = torch.searchsorted(table, v.contiguous()).clamp(1, table.numel() - 1)
    down, up = v - table[hi - 1], table[hi] - v
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def _decoded64(byte, d, q, bits):
    """Values of quantised rows, byte by byte."""
    e2m1, e4m3 = _tables64()
    n = byte.long()
    f8 = lambda c: e4m3[(c & 127).clamp(max=126)] * (1 - 2 * (c >> 7))  # noqa: E731
    at, tail = q if bits == 8 else q // 2 + q // 16, _tail_at(q, bits)
    word = (n[:, at : at + 4] << torch.tensor([0, 8, 16, 24], device=DEV)).sum(1)
    s = 2.0 ** ((word >> 23) - 127).double()[:, None]
    if bits == 8:
        v = f8(n[:, :q]) * s
    else:
        c = torch.arange(q, device=DEV)
        half = (n[:, c // 2] >> (4 * (c % 2))) & 15
        v = e2m1[half & 7] * (1 - 2 * (half >> 3)) * f8(n[:, q // 2 + c // 16]) * s
    rest = n[:, tail : tail + 2 * (d - q)]
    rest = (rest[:, 0::2] + 256 * rest[:, 1::2]).to(torch.int32) << 16
    return torch.cat([v, rest.view(torch.float32).double()], 1)


def _exact_write(case, s):
    q, bits = case["Q"], case["bits"]
    e2m1, e4m3 = _tables64()
    x = s["x"].double()
    v = x[:, :q].clone()
    most = v.abs().amax(1)
    s_ = torch.full_like(most, 2.0 ** -48)
    for e in range(-48, 49):  # the smallest power of two that is enough
        s_ = torch.where(s_ * (448 if bits == 8 else 2688) < most, 2.0 ** e, s_)
    v = v / s_[:, None]
    sign = torch.where(v < 0, -1.0, 1.0).double()
    if bits == 8:
        v = sign * e4m3[_nearest(v.abs(), e4m3)]
    else:
        block = e4m3[_nearest(v.abs().reshape(-1, q // 16, 16).amax(2) / 6, e4m3)].repeat_interleave(16, 1)
        v = sign * e2m1[_nearest(v.abs() / torch.where(block > 0, block, torch.inf), e2m1)] * block
    return torch.cat([v * s_[:, None], x[:, q:]], 1)


def _exact_mla(case, s):
    b, nq, h, d, k, page = (case[x] for x in ("B", "nq", "H", "D", "K", "page"))
    lens, table = s["seq_lens"].tolist(), s["table"].long()
    rows = s["cache"].reshape(-1, s["cache"].shape[2])
    outs, lses = [], []
    for r in range(b):
        for j in range(nq):
            n = r * nq + j
            v = max(0, lens[r] - nq + j + 1)
            at = torch.arange(v, device=DEV)
            if k:
                at = s["topk_idx"][n].long()
                at = at[at >= 0]
            kv = _decoded64(rows[table[r][at // page] * page + at % page], d, DV, case["bits"])
            z = (s["q"][n].double() @ kv.T) * s["scale"]
            every = z if s["sink"] is None else torch.cat([z, s["sink"].double()[:, None]], 1)
            if every.shape[1] == 0:
                outs.append(torch.zeros(h, DV, dtype=torch.float64, device=DEV))
                lses.append(torch.full((h,), -math.inf, dtype=torch.float64, device=DEV))
                continue
            lse = torch.logsumexp(every, 1)
            outs.append(torch.exp(z - lse[:, None]) @ kv[:, :DV])
            lses.append(lse)
    return torch.stack(outs), torch.stack(lses)


def exact(case, seed):
    op = case["op"]
    if op == "write":
        return _exact_write(case, prepare(case, seed))
    lens = _contexts(case)
    if op == "read":
        s = prepare(case, seed)
        page, table = case["page"], s["table"].long()
        at = [table[i][p // page] * page + p % page for i, n in enumerate(lens) for p in [torch.arange(n, device=DEV)]]
        return _decoded64(s["cache"].reshape(-1, s["cache"].shape[2])[torch.cat(at)], case["D"], case["Q"], case["bits"])
    if sum(lens) * case["nq"] * case["H"] > 1 << 27 or case["B"] * case["nq"] > 512:
        return None
    return _exact_mla(case, prepare(case, seed))
