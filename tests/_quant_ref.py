"""Rows of a quantised cache in plain 64-bit arithmetic, from the description of the format (torch on the CPU)."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.tensor([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127],
                    dtype=torch.float64)


def layout(D, Q, bits):
    """(offset of the block scales, of s, of the other channels, bytes of a row)."""
    blocks = Q if bits == 8 else Q // 2
    s = blocks if bits == 8 else blocks + Q // 16
    up = lambda n: (n + 15) // 16 * 16  # noqa: E731
    return blocks, s, up(s + 4), up(s + 4) + up(2 * (D - Q))


def nearest(v, table):
    """Index of the nearest entry for magnitudes v, ties to the even index; past the table its last entry."""
    d = (v[..., None] - table).abs()
    best = d.min(-1).values
    i = torch.arange(len(table)).expand(d.shape)
    first = torch.where(d == best[..., None], i, 999).min(-1).values
    last = torch.where(d == best[..., None], i, -1).max(-1).values
    return torch.where(first % 2 == 0, first, last)


def encode(x, Q, bits):
    """Bytes uint8 [T, row bytes] of bf16 rows x [T, D]."""
    T, D = x.shape
    blocks, at, tail, width = layout(D, Q, bits)
    out = torch.zeros(T, width, dtype=torch.uint8)
    v = x[:, :Q].double()
    for t in range(T):
        a, most = v[t], v[t].abs().max()
        fits = [e for e in range(-48, 49) if most <= (448 if bits == 8 else 2688) * 2.0 ** e]
        s = 2.0 ** fits[0] if bool(torch.isfinite(a).all()) and fits else float("nan")
        out[t, at:at + 4] = torch.tensor([s], dtype=torch.float32).view(torch.uint8)
        out[t, tail:tail + 2 * (D - Q)] = x[t, Q:].contiguous().view(torch.uint8)
        if s != s:
            continue
        if bits == 8:
            out[t, :Q] = (nearest(a.abs() / s, E4M3) + 128 * torch.signbit(a)).to(torch.uint8)
            continue
        b = nearest(a.abs().reshape(-1, 16).max(1).values / (6 * s), E4M3)
        scale = E4M3[b].repeat_interleave(16)
        c = nearest(a.abs() / torch.where(scale > 0, scale * s, torch.inf), E2M1) + 8 * torch.signbit(a)
        out[t, :Q // 2] = (c[0::2] + 16 * c[1::2]).to(torch.uint8)
        out[t, blocks:at] = b.to(torch.uint8)
    return out


def decode(rows, D, Q, bits):
    """Values fp64 [T, D] of rows uint8 [T, row bytes]."""
    rows = rows.cpu()
    blocks, at, tail, _ = layout(D, Q, bits)
    s = rows[:, at:at + 4].contiguous().view(torch.float32).double()
    n = rows.long()
    signed = lambda mag, sign: torch.where(sign > 0, -mag, mag)  # noqa: E731
    if bits == 8:
        v = signed(E4M3[(n[:, :Q] & 127).clamp(max=126)], n[:, :Q] >> 7)
    else:
        c = torch.stack([n[:, :Q // 2] & 15, n[:, :Q // 2] >> 4], -1).flatten(1)
        v = signed(E2M1[c & 7], c >> 3) * E4M3[(n[:, blocks:at] & 127).clamp(max=126)].repeat_interleave(16, 1)
    return torch.cat([v * s, rows[:, tail:tail + 2 * (D - Q)].contiguous().view(torch.bfloat16).double()], 1)


def attention(q, cache, bits, table, seq_lens, cu_q, scale, sink=None, topk=None, topk_len=None):
    """out [N, H, 512], lse [N, H] in 64 bits (NaN outside the requests), and per row what bounds a kernel's error:
    size [N, H] = the largest scale * sum |q k| over the positions seen, mass [N, H, 512] = sum of weights * |kv|,
    top [N, H, 512] = (the largest weight times its row's s) * sum of |kv| / s, and most [N, H] = the largest scale * (largest
    |q| of the first 512 channels) * sum of their |k|."""
    N, H, D = q.shape
    page = cache.shape[1]
    flat = cache.cpu().reshape(-1, cache.shape[2])
    nan = float("nan")
    out, mass = torch.full((N, H, 512), nan, dtype=torch.float64), torch.zeros(N, H, 512, dtype=torch.float64)
    lse, size = torch.full((N, H), nan, dtype=torch.float64), torch.zeros(N, H, dtype=torch.float64)
    top, most, at_s = torch.zeros_like(mass), torch.zeros_like(size), layout(D, 512, bits)[1]
    for b in range(len(seq_lens)):
        lo, hi = cu_q[b], cu_q[b + 1]
        for n in range(lo, hi):
            v = max(0, seq_lens[b] - (hi - lo) + (n - lo) + 1)
            at = list(range(v))
            if topk is not None:
                keep = topk[n].tolist() if topk_len is None else topk[n].tolist()[:max(0, int(topk_len[n]))]
                at = [i for i in keep if 0 <= i < v]
            rows = [int(table[b][p // page]) * page + p % page for p in at]
            kv = decode(flat[rows], D, 512, bits) if rows else torch.zeros(0, D, dtype=torch.float64)
            z = (q[n].double() @ kv.T) * scale
            full = z if sink is None else torch.cat([z, sink.double()[:, None]], 1)
            if full.shape[1] == 0:
                out[n], lse[n] = 0.0, -float("inf")
                continue
            lse[n] = torch.logsumexp(full, 1)
            p = torch.exp(z - torch.where(torch.isinf(lse[n]), torch.zeros(()).double(), lse[n])[:, None])
            out[n], mass[n] = p @ kv[:, :512], p @ kv[:, :512].abs()
            if rows:
                size[n] = (q[n].double().abs() @ kv.abs().T).max(1).values * scale
                s = flat[rows][:, at_s:at_s + 4].contiguous().view(torch.float32).double()[:, 0]
                s = torch.where(s < 2.0 ** -48, 2.0 ** -48, s)  # (a row that was never written)
                top[n] = (p * s).max(1, keepdim=True).values * (kv[:, :512].abs() / s[:, None]).sum(0)
                most[n] = q[n, :, :512].double().abs().max(1).values * float(kv[:, :512].abs().sum(1).max()) * scale
    return out, lse, size, mass, top, most


def check_attention(got, want, bits):
    """out and lse of a kernel against attention()'s answer; rows that are NaN there are not looked at.

    A score is a sum of 576 exact products in fp32.  Whether they are added one by one, by sixteens or in a tree, and by
    truncation or to nearest, its error is at most 80 * 2^-23 times the sum of magnitudes, times the scale: dz.  With 8 bits
    a query is two numbers of 4 bits, which leaves up to 2^-17 of its row's largest channel of each channel.  Forming 2^x
    from a score adds 2^-21 of a weight, and 2^-23 of x, |x| being at most twice size.

    4 bits: a weight is rounded to 11 bits (2^-11), and where it is below 2^-14 to a multiple of 2^-24, the largest weight
    times its row's s being 2^7 at least: that is 2^-32 of it times |kv| / s of each position at most.
    8 bits: to 3 bits, which leaves 2^-3 of its power of two at most, and what is left to 4 bits (2^-7 of the weight) or,
    below 2^-6, to a multiple of 2^-9 (2^-10), the largest weight times its row's s being 2^5 at least: 2^-15 of it.

    A sum of weights or products in fp32 adds less than 2^-13 of its mass at the lengths tested; the output is rounded to
    bf16 (2^-8 of it)."""
    out, lse, size, mass, top, most = want
    o, l = got[0].cpu().double(), got[1].cpu().double()
    seen = ~torch.isnan(lse)
    dz = 84 * 2.0 ** -23 * size + 2.0 ** -20 + (2.0 ** -17 * most if bits == 8 else 0.0)
    fin = seen & torch.isfinite(lse)
    assert torch.equal(torch.isinf(l) & seen, torch.isinf(lse) & seen)
    assert bool(((l - lse).abs() <= dz + 2.0 ** -13 + 2.0 ** -22 * lse.abs())[fin].all())
    w, floor = (2.0 ** -7, 2.0 ** -15) if bits == 8 else (2.0 ** -11, 2.0 ** -32)
    tol = 2.0 ** -8 * out.abs() + (w + 2.0 ** -13 + 2 * dz)[..., None] * mass + floor * top + 2.0 ** -133
    assert bool((o - out).abs()[seen].le(tol[seen]).all()), float(((o - out).abs() / tol)[seen].max())
