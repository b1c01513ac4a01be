"""Plain 64-bit forms of the serving step's operators (numpy / torch on the CPU), for the parity tests."""
import numpy as np
import torch


def slots(seq_lens, new_lens, table, free, page, N):
    """Request by request, token by token; None when the step does not fit."""
    B = len(seq_lens)
    new = [1] * B if new_lens is None else list(new_lens)
    table = [list(r) for r in table]
    taken, slot_map, pos, cu = 0, [], [], [0]
    for b in range(B):
        s, n = seq_lens[b], new[b]
        if s < 0 or n < 0 or -(-(s + n) // page) > len(table[b]):
            return None
        for j in range(n):
            p = s + j
            if p % page == 0:
                if taken >= len(free):
                    return None
                table[b][p // page] = free[taken]
                taken += 1
            slot_map.append(table[b][p // page] * page + p % page)
            pos.append(p)
        cu.append(cu[-1] + n)
    if cu[-1] > N:
        return None
    pad = [-1] * (N - cu[-1])
    return slot_map + pad, pos + pad, cu, [s + n for s, n in zip(seq_lens, new)], taken, table


def _pairs(r0, R, inter):
    i = np.arange(R // 2)
    return (r0 + 2 * i, r0 + 2 * i + 1) if inter else (r0 + i, r0 + R // 2 + i)


def _turn(v, pos, inv_freq, r0, inter, scale, sign):
    """v [T, H, D] fp64 with its rotated channels multiplied by scale exp(sign i angle)."""
    if inv_freq is None or len(inv_freq) == 0:
        return v
    a, b = _pairs(r0, 2 * len(inv_freq), inter)
    ang = pos[:, None, None] * inv_freq[None, None, :]
    w = (v[..., a] + 1j * v[..., b]) * np.exp(sign * 1j * ang) * scale
    v = v.copy()
    v[..., a], v[..., b] = w.real, w.imag
    return v


def _hat(x, kind, n, eps):
    u = x[..., :n]
    if kind == "layer":
        u = u - u.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    return u * r, r


def norm_rope_fwd(x, kind, n, w, b, eps, pos, inv_freq, r0, inter, scale=1.0):
    y = x.copy()
    if kind != "none":
        hat, _ = _hat(x, kind, n, eps)
        y[..., :n] = hat * (1.0 if w is None else w) + (0.0 if b is None else b)
    return _turn(y, pos, inv_freq, r0, inter, scale, 1)


def norm_rope_bwd(g, x, kind, n, w, eps, pos, inv_freq, r0, inter, scale=1.0):
    """dx, dw, db, the sums of |terms| that bound the rounding of dw and db, and the largest of the terms whose
    difference dx is, per row."""
    g = _turn(g, pos, inv_freq, r0, inter, scale, -1)
    most = np.abs(g).max(-1, keepdims=True)
    if kind == "none":
        return g, None, None, None, None, most
    hat, r = _hat(x, kind, n, eps)
    gy = g[..., :n]
    gw = gy * (1.0 if w is None else w)
    d = gw - hat * (gw * hat).mean(-1, keepdims=True)
    if kind == "layer":
        d = d - gw.mean(-1, keepdims=True)
    dx = g.copy()
    dx[..., :n] = r * d
    part = np.abs(gw) + np.abs(hat) * np.abs(gw * hat).mean(-1, keepdims=True) + np.abs(gw).mean(-1, keepdims=True)
    most = np.maximum(most, (r * part).max(-1, keepdims=True))
    return dx, (gy * hat).sum((0, 1)), gy.sum((0, 1)), np.abs(gy * hat).sum((0, 1)), np.abs(gy).sum((0, 1)), most


def rows_of(table_row, positions, page):
    return [int(table_row[p // page]) * page + p % page for p in positions]


def visible(seq_len, n_new, j):
    """Positions that new token j of n_new sees."""
    return max(0, seq_len - n_new + j + 1)


def paged_mla(q, cache, table, seq_lens, cu_q, scale, page, sink=None, topk=None, topk_len=None):
    """out [N, H, 512], lse [N, H] in 64 bits; rows outside every request are NaN."""
    N, H, D = q.shape
    rows = cache.double().reshape(-1, D)
    out = torch.full((N, H, 512), float("nan"), dtype=torch.float64)
    lse = torch.full((N, H), float("nan"), dtype=torch.float64)
    for b in range(len(seq_lens)):
        lo, hi = cu_q[b], cu_q[b + 1]
        for n in range(lo, hi):
            v = visible(seq_lens[b], hi - lo, n - lo)
            at = list(range(v))
            if topk is not None:
                keep = topk[n].tolist() if topk_len is None else topk[n].tolist()[:max(0, int(topk_len[n]))]
                at = [i for i in keep if 0 <= i < v]
            kv = rows[rows_of(table[b], at, page)]
            z = (q[n].double() @ kv.T) * scale
            full = z if sink is None else torch.cat([z, sink.double()[:, None]], 1)
            if full.shape[1] == 0:
                out[n], lse[n] = 0.0, -float("inf")
                continue
            lse[n] = torch.logsumexp(full, 1)
            p = torch.exp(z - torch.where(torch.isinf(lse[n]), torch.zeros(()).double(), lse[n])[:, None])
            out[n] = p @ kv[:, :512]
    return out, lse


def paged_scores(q, cache, w, table_row, v, page):
    """Indexer scores of one token over its v visible positions, and their magnitude sum."""
    rows = cache.double().reshape(-1, q.shape[-1])[rows_of(table_row, range(v), page)]
    d = q.double() @ rows.T
    m = q.double().abs() @ rows.abs().T
    return (w.double()[:, None] * d.clamp(min=0)).sum(0), (w.double().abs()[:, None] * m).sum(0)


def topk_of(scores, K):
    """The K best positions (ties to the lower), ascending."""
    order = sorted(range(len(scores)), key=lambda i: (-float(scores[i]), i))[:K]
    return sorted(order)
