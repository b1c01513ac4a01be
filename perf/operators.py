"""The operators of the serving step around the sparse attention, in their plain form and through the framework.

Four operators: the slots of a step's new tokens (``dsa_paged_slots``), the normalisation of a row with the
rotation of its positions and their gradient (``dsa_norm_rope_fwd`` / ``dsa_norm_rope_bwd``), the attention of new
tokens over a paged latent cache (``dsa_paged_mla``), and the selection over paged index keys
(``dsa_paged_indexer_topk``)."""
import math

import numpy as np
import torch

own = False

DV = 512
DEV = "cuda"


# ----------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a full batch: one new token for each of 256 requests
        {"name": "slots, decode of 256", "op": "slots", "B": 256, "ctx": 30000, "new": 1, "page": 64},
        # a step that takes in prompts of very different lengths
        {"name": "slots, prompts of 48", "op": "slots", "B": 48, "ctx": 5000, "new": 5321, "page": 64},
        # the latents of a decode step: RMS norm of 512 channels, rotation of 64, written to their cache slots
        {"name": "latents to the cache, 32", "op": "fwd", "T": 32, "H": 1, "D": 576, "norm": "rms", "norm_dim": 512,
         "rope": 64, "rope_start": 512, "inter": True, "wide": 0, "slots": True, "far": 32768},
        # a training step's query heads: only the 64 position channels of 576 are turned, heads of a wider row
        {"name": "query positions, 16384 x 64", "op": "fwd", "T": 16384, "H": 64, "D": 64, "norm": "none",
         "norm_dim": 0, "rope": 64, "rope_start": 0, "inter": True, "wide": 512, "slots": False, "far": 131072},
        # per-head norm of queries with the rotation of half the head
        {"name": "head norm, 4097 x 32 x 128", "op": "fwd", "T": 4097, "H": 32, "D": 128, "norm": "rms",
         "norm_dim": 128, "rope": 64, "rope_start": 0, "inter": False, "wide": 0, "slots": False, "far": 1000000},
        # gradient of the index keys' layer norm and rotation, one 32k sequence
        {"name": "index keys' gradient, 32768", "op": "bwd", "T": 32768, "H": 1, "D": 128, "norm": "layer",
         "norm_dim": 128, "rope": 64, "rope_start": 0, "inter": False, "wide": 0, "slots": False, "far": 32768},
        # the smallest attention call: one request, a short context, a few local heads
        {"name": "attention, 1 x 1000, 16 heads", "op": "mla", "B": 1, "L": 1000, "H": 16, "nq": 1, "D": 576,
         "page": 16, "K": 0, "sink": False},
        # a serving batch of mixed lengths
        {"name": "attention, 64 x 16k, 64 heads", "op": "mla", "B": 64, "L": 16384, "H": 64, "nq": 1, "D": 576,
         "page": 64, "K": 0, "sink": False},
        # one long context with all the heads on one GPU, two tokens (one drafted)
        {"name": "attention, 1 x 131k, 128 heads", "op": "mla", "B": 1, "L": 131071, "H": 128, "nq": 2, "D": 576,
         "page": 64, "K": 0, "sink": False},
        # the sparse form: every token attends to its own 2048 selected positions
        {"name": "attention, 48 x 2048 selected", "op": "mla", "B": 48, "L": 20000, "H": 64, "nq": 1, "D": 576,
         "page": 64, "K": 2048, "sink": True},
        # selection for one long request: latency
        {"name": "selection, 1 x 65k", "op": "topk", "B": 1, "L": 65001, "Hi": 64, "nq": 1, "page": 64, "K": 2048},
        # selection for a batch with one drafted token each
        {"name": "selection, 32 x 32k", "op": "topk", "B": 32, "L": 32768, "Hi": 64, "nq": 2, "page": 64, "K": 2048},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["slots", "fwd", "bwd", "mla", "mla", "topk"])
    if op == "slots":
        b = _log(rng, 1, 1024)
        return {"op": op, "B": b, "ctx": _log(rng, 1, 60000), "new": _log(rng, 1, max(1, min(8192, 131072 // b))),
                "page": rng.choice([1, 16, 33, 64, 128])}
    if op in ("fwd", "bwd"):
        d, nd, r, r0 = rng.choice([(576, 512, 64, 512), (128, 128, 64, 0), (128, 128, 128, 0), (192, 0, 64, 128),
                                   (80, 80, 40, 8), (64, 0, 64, 0), (97, 97, 30, 67)])
        h = 1 if d == 576 else rng.choice([1, 4, 24, 64])
        norm = rng.choice(["rms", "layer"]) if nd else "none"
        return {"op": op, "T": _log(rng, 1, (1 << 26) // (h * d * (2 if op == "bwd" else 1))), "H": h, "D": d,
                "norm": norm, "norm_dim": nd, "rope": r, "rope_start": r0, "inter": rng.random() < 0.5,
                "wide": rng.choice([0, 0, 64]), "slots": op == "fwd" and h == 1 and rng.random() < 0.5,
                "far": _log(rng, 100, 1000000)}
    b, nq, page = _log(rng, 1, 128), rng.choice([1, 1, 2, 4]), rng.choice([16, 48, 64, 128])
    if op == "mla":
        h = rng.choice([1, 5, 8, 16, 24, 40, 64, 128])
        k = rng.choice([0, 0, _log(rng, 1, 2048)])
        return {"op": op, "B": b, "L": _log(rng, 1, min(131072, 524288 // b, (1 << 25) // (b * nq * h))), "H": h,
                "nq": nq, "D": rng.choice([512, 576]), "page": page, "K": k, "sink": rng.random() < 0.3}
    hi = rng.choice([4, 8, 32, 64])
    long = _log(rng, 40, min(131072, 524288 // b, (1 << 26) // (b * nq * hi)))
    return {"op": op, "B": b, "L": long, "Hi": hi, "nq": nq, "page": page, "K": _log(rng, 1, min(2048, long // 2))}


def _lens(b, most):
    """Mixed lengths from about a quarter of the longest up to it, the same for every seed."""
    f = [((i + 1) * 0.6180339887498949) % 1.0 for i in range(b)]
    return [most if i == 0 else max(1, int(most * (0.25 + 0.75 * f[i]))) for i in range(b)]


def _contexts(case):
    """Lengths of the requests, new tokens included; now and then fewer than the new tokens (rows that see nothing)."""
    return [n if i % 5 == 3 else max(n, case["nq"]) for i, n in enumerate(_lens(case["B"], case["L"]))]


def _news(case):
    if case["new"] == 1:
        return [1] * case["B"]
    return [max(0, x - case["new"] // 5) for x in _lens(case["B"], case["new"])]


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pages(lens, page, g, spare):
    """A table of randomly placed pages for requests of these lengths, and the pages that are left."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    wide = max(need) if need else 1
    table = torch.full((len(lens), max(1, wide)), -1, dtype=torch.int32, device=DEV)
    counts = torch.tensor(need, device=DEV)
    cols = torch.arange(max(1, wide), device=DEV)[None, :]
    table[cols < counts[:, None]] = perm[: sum(need)]
    return table, perm[sum(need):].contiguous(), total


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    randn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    if op == "slots":
        news = _news(case)
        off = int(torch.randint(0, max(1, case["ctx"]), (1,), generator=g, device=DEV))
        ctx = [(n + off * (i + 1)) % case["ctx"] for i, n in enumerate(_lens(case["B"], case["ctx"]))]
        page = case["page"]
        fresh = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, news))
        table, free, _ = _pages(ctx, page, g, fresh + 1000)
        most = -(-(case["ctx"] + max(news)) // page) + 1
        wide = torch.full((case["B"], most), -1, dtype=torch.int32, device=DEV)
        wide[:, : table.shape[1]] = table
        s.update(seq_lens=_ints(ctx), new_lens=_ints(news), table=wide, N=sum(news) + 3, free=free)
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device=DEV)
        return s
    if op in ("fwd", "bwd"):
        t, h, d = case["T"], case["H"], case["D"]
        rows = lambda: randn(t, h, case["wide"] + d).bfloat16()[..., case["wide"]:]  # noqa: E731
        s["x"] = rows()
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV).to(torch.int32)
        i = torch.arange(case["rope"] // 2, dtype=torch.float64, device=DEV)
        s["inv_freq"] = (10000.0 ** (-2.0 * i / case["rope"])).float()
        nd = case["norm_dim"]
        s["weight"] = 1 + 0.2 * randn(nd) if nd else None
        s["bias"] = 0.2 * randn(nd) if case["norm"] == "layer" else None
        if case["slots"]:
            n = 2 * t + 64
            s["cache"] = torch.zeros(n, h, d, dtype=torch.bfloat16, device=DEV)
            rows_ = torch.randperm(n, generator=g, device=DEV)[:t].to(torch.int32)
            rows_[5::97] = -1  # padding of a captured batch
            s["rows"] = rows_
        else:
            s["out"] = torch.empty(t, h, d, dtype=torch.bfloat16, device=DEV)
        if op == "bwd":
            s["dout"] = randn(t, h, d).bfloat16()
        if own:
            import sparse_attention_mla_gb300 as dsa

            kind = "norm_rope_bwd" if op == "bwd" else "norm_rope_fwd"
            s["ws"] = torch.zeros(dsa.paged_workspace_size(kind, t * h, nd), dtype=torch.uint8, device=DEV)
        return s
    b, nq, page = case["B"], case["nq"], case["page"]
    lens = _contexts(case)
    table, _, total = _pages(lens, page, g, 4)
    s.update(seq_lens=_ints(lens), table=table, cu_q=_ints([i * nq for i in range(b + 1)]))
    n = b * nq
    if op == "mla":
        h, d = case["H"], case["D"]
        s["q"] = randn(n, h, d).bfloat16()
        s["cache"] = randn(total, page, d).bfloat16()
        s["scale"] = d ** -0.5 * 1.7
        s["sink"] = randn(h) if case["sink"] else None
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
        kind, args = "mla", (n, h)
    else:
        hi = case["Hi"]
        # values of a quantised indexer: multiples of 1/8, weights multiples of 1/1024 (every sum is exact)
        grid = lambda x: ((x * 8).round() / 8).clamp(-3, 3).bfloat16()  # noqa: E731
        s["q"] = grid(randn(n, hi, 128))
        s["cache"] = grid(randn(total, page, 128))
        s["w"] = (torch.rand(n, hi, generator=g, device=DEV) * 128).round() / 1024
        s["topk_idx"] = torch.empty(n, case["K"], dtype=torch.int32, device=DEV)
        s["topk_len"] = torch.empty(n, dtype=torch.int32, device=DEV)
        kind, args = "topk", (n, table.shape[1] * page)
    if own:
        import sparse_attention_mla_gb300 as dsa

        s["ws"] = torch.zeros(dsa.paged_workspace_size(kind, *args), dtype=torch.uint8, device=DEV)
    return s


def _visible(s):
    """Positions that each query token sees (its own included)."""
    nq = s["nq"]
    j = torch.arange(nq, device=DEV)
    return (s["seq_lens"].long()[:, None] - nq + j[None, :] + 1).clamp(min=0).reshape(-1)


# ------------------------------------------------------------------------------------------------- plain forms
def _slots_plain(s):
    page, n_max = s["page"], s["N"]
    old, new = s["seq_lens"].long(), s["new_lens"].long()
    b = old.numel()
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    cu = torch.cat([zero, torch.cumsum(new, 0)])
    first = (old + page - 1) // page
    taken = (old + new + page - 1) // page - first
    base = torch.cat([zero, torch.cumsum(taken, 0)])
    cols = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    fresh = (cols >= first[:, None]) & (cols < (first + taken)[:, None])
    at = (base[:b, None] + cols - first[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    t = torch.arange(n_max, device=DEV)
    r = torch.searchsorted(cu, t, right=True) - 1
    real = t < cu[b]
    r = r.clamp(0, b - 1)
    pos = old[r] + t - cu[r]
    page_of = table[r, (pos // page).clamp(0, table.shape[1] - 1)].long()
    slot = torch.where(real, page_of * page + pos % page, -1)
    pos = torch.where(real, pos, -1)
    i32 = torch.int32
    return {"table": table, "slots": slot.to(i32), "positions": pos.to(i32), "cu": cu.to(i32),
            "seq_lens": (old + new).to(i32), "taken": base[b:].to(i32)}


def _cos_sin(s, dtype):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    return torch.cos(angle).to(dtype)[:, None, :], torch.sin(angle).to(dtype)[:, None, :]


def _halves(s, r):
    if s["inter"]:
        return r[..., 0::2], r[..., 1::2]
    return r[..., : s["rope"] // 2], r[..., s["rope"] // 2:]


def _joined(s, a, b):
    return torch.stack([a, b], -1).flatten(-2) if s["inter"] else torch.cat([a, b], -1)


def _norm_parts(s, x):
    """The normalised channels before the weight, and what they were divided by."""
    nd = s["norm_dim"]
    u = x[..., :nd]
    if s["norm"] == "layer":
        u = u - u.mean(-1, keepdim=True)
    r = torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6)
    return u * r, r


def _fwd_values(s, dtype):
    x = s["x"].to(dtype)
    nd, r0, r1 = s["norm_dim"], s["rope_start"], s["rope_start"] + s["rope"]
    if nd:
        y, _ = _norm_parts(s, x)
        y = y * s["weight"].to(dtype)
        if s["bias"] is not None:
            y = y + s["bias"].to(dtype)
        x = torch.cat([y, x[..., nd:]], -1)
    c, sn = _cos_sin(s, dtype)
    a, b = _halves(s, x[..., r0:r1])
    return torch.cat([x[..., :r0], _joined(s, a * c - b * sn, b * c + a * sn), x[..., r1:]], -1)


def _fwd_plain(s):
    y = _fwd_values(s, torch.float32).bfloat16()
    if not s["slots"]:
        return y
    keep = s["rows"] >= 0
    s["cache"][s["rows"][keep].long()] = y[keep]
    return s["cache"]


def _bwd_values(s, dtype):
    g, x = s["dout"].to(dtype), s["x"].to(dtype)
    nd, r0, r1 = s["norm_dim"], s["rope_start"], s["rope_start"] + s["rope"]
    c, sn = _cos_sin(s, dtype)
    a, b = _halves(s, g[..., r0:r1])
    g = torch.cat([g[..., :r0], _joined(s, a * c + b * sn, b * c - a * sn), g[..., r1:]], -1)
    if not nd:
        return g, None, None
    xh, r = _norm_parts(s, x)
    gy = g[..., :nd]
    dw = (gy * xh).double().sum((0, 1))
    db = gy.double().sum((0, 1)) if s["bias"] is not None else None
    gw = gy * s["weight"].to(dtype)
    d = gw - xh * (gw * xh).mean(-1, keepdim=True)
    if s["norm"] == "layer":
        d = d - gw.mean(-1, keepdim=True)
    return torch.cat([d * r, g[..., nd:]], -1), dw, db


def _bwd_plain(s):
    dx, dw, db = _bwd_values(s, torch.float32)
    f32 = lambda v: None if v is None else v.float()  # noqa: E731
    return dx.bfloat16(), f32(dw), f32(db)


def _row_numbers(s, pos):
    """Cache rows [B, S] of positions [B, S] (in range)."""
    page = s["page"]
    return torch.gather(s["table"].long(), 1, pos // page) * page + pos % page


def _mla_plain(s):
    b, nq, h, d = s["B"], s["nq"], s["H"], s["D"]
    rows = s["cache"].reshape(-1, d)
    q = s["q"].float().reshape(b, nq * h, d) * s["scale"]
    vis = _visible(s)
    if s["K"]:
        idx = s["topk_idx"].long().reshape(b, nq * s["K"])
        kv = rows[_row_numbers(s, idx.clamp(min=0))].float().reshape(b * nq, s["K"], d)
        z = torch.matmul(q.reshape(b * nq, h, d), kv.transpose(1, 2))
        seen = (s["topk_idx"] >= 0)[:, None, :]
    else:
        most = s["table"].shape[1] * s["page"]
        pos = torch.arange(most, device=DEV)[None, :].expand(b, most)
        pos = torch.minimum(pos, (s["seq_lens"].long() - 1)[:, None])
        kv = rows[_row_numbers(s, pos)].float()
        z = torch.matmul(q, kv.transpose(1, 2)).reshape(b * nq, h, most)
        seen = (torch.arange(most, device=DEV)[None, :] < vis[:, None])[:, None, :]
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
    if s["K"]:
        out = torch.matmul(p, kv[..., :DV])
    else:
        out = torch.matmul(p.reshape(b, nq * h, -1), kv[..., :DV]).reshape(b * nq, h, DV)
    return out.bfloat16(), lse


def _topk_plain(s):
    b, nq, hi, k = s["B"], s["nq"], s["Hi"], s["K"]
    rows = s["cache"].reshape(-1, 128)
    most = s["table"].shape[1] * s["page"]
    pos = torch.arange(most, device=DEV)[None, :].expand(b, most)
    pos = torch.minimum(pos, (s["seq_lens"].long() - 1)[:, None])
    keys = rows[_row_numbers(s, pos)].float()
    dots = torch.matmul(s["q"].float().reshape(b, nq * hi, 128), keys.transpose(1, 2)).clamp_(min=0)
    score = torch.matmul(s["w"].reshape(b * nq, 1, hi), dots.reshape(b * nq, hi, most))[:, 0]
    vis = _visible(s)
    seen = torch.arange(most, device=DEV)[None, :] < vis[:, None]
    score = torch.where(seen, score, -torch.inf)
    order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :k]
    cnt = vis.clamp(max=k)
    taken = torch.arange(order.shape[1], device=DEV)[None, :] < cnt[:, None]
    order = torch.sort(torch.where(taken, order, most), dim=1).values
    idx = torch.full((b * nq, k), -1, dtype=torch.int32, device=DEV)
    idx[:, : order.shape[1]] = torch.where(order < most, order, -1).to(torch.int32)
    return idx, cnt.to(torch.int32)


# ------------------------------------------------------------------------------------------------------- a pass
def run(s):
    op = s["op"]
    if not own:
        if op == "slots":
            return _slots_plain(s)
        if op == "fwd":
            return _fwd_plain(s)
        if op == "bwd":
            return _bwd_plain(s)
        return _mla_plain(s) if op == "mla" else _topk_plain(s)
    import sparse_attention_mla_gb300 as dsa

    if op == "slots":
        slots, pos, cu, seq_lens, taken = dsa.dsa_paged_slots(
            s["seq_lens"], s["table"], s["free"], s["page"], new_lens=s["new_lens"], N=s["N"], workspace=s["ws"])
        return {"table": s["table"], "slots": slots, "positions": pos, "cu": cu, "seq_lens": seq_lens, "taken": taken}
    if op in ("fwd", "bwd"):
        args = dict(inv_freq=s["inv_freq"], positions=s["positions"], norm=s["norm"], norm_dim=s["norm_dim"],
                    weight=s["weight"], eps=1e-6, rope_start=s["rope_start"], interleaved=s["inter"], workspace=s["ws"])
        if op == "bwd":
            return dsa.dsa_norm_rope_bwd(s["dout"], s["x"], with_bias=s["bias"] is not None, **args)
        if s["slots"]:
            return dsa.dsa_norm_rope_fwd(s["x"], bias=s["bias"], out=s["cache"], out_rows=s["rows"], **args)
        return dsa.dsa_norm_rope_fwd(s["x"], bias=s["bias"], out=s["out"], **args)
    if op == "mla":
        return dsa.dsa_paged_mla(s["q"], s["cache"], s["table"], s["seq_lens"], s["scale"], cu_q=s["cu_q"],
                                 topk_idx=s.get("topk_idx"), topk_len=s.get("topk_len"), attn_sink=s["sink"],
                                 out=s["out"], lse=s["lse"], workspace=s["ws"])
    return dsa.dsa_paged_indexer_topk(s["q"], s["cache"], s["w"], s["table"], s["seq_lens"], s["K"], cu_q=s["cu_q"],
                                      topk_idx=s["topk_idx"], topk_len=s["topk_len"], workspace=s["ws"])


def work(case):
    op = case["op"]
    if op == "slots":
        b, n = case["B"], sum(_news(case))
        fresh = n // case["page"] + b
        return {"bytes": 4 * (2 * b + 2 * fresh + 2 * b + 2 * n), "flops": 4 * n}
    if op in ("fwd", "bwd"):
        n = case["T"] * case["H"] * case["D"]
        moved = 4 * n + 4 * case["T"] if op == "fwd" else (6 if case["norm_dim"] else 4) * n
        return {"bytes": moved + 8 * case["norm_dim"] + 4 * case["T"], "flops": (8 if op == "fwd" else 16) * n}
    b, nq = case["B"], case["nq"]
    lens = _contexts(case)
    vis = [max(0, n - nq + j + 1) for n in lens for j in range(nq)]
    if op == "mla":
        h, d, k = case["H"], case["D"], case["K"]
        pairs = sum(min(v, k) for v in vis) if k else sum(vis)
        rows = min(pairs, sum(lens)) if k else sum(lens)
        moved = rows * d * 2 + b * nq * h * (2 * d + 2 * DV + 4) + (4 * b * nq * k)
        return {"bytes": moved, "flops": 2 * h * (d + DV) * pairs}
    moved = sum(lens) * 256 + b * nq * (case["Hi"] * 260 + 4 * case["K"])
    return {"bytes": moved, "flops": 2 * case["Hi"] * 128 * sum(vis)}


# ------------------------------------------------------------------------------- 64 bits, from the definitions
def _rotated64(case, v, pos, inv_freq, sign):
    """Channels [rope_start, rope_start + rope) as complex numbers times exp(sign i angle)."""
    r0, r = case["rope_start"], case["rope"]
    at = np.arange(r // 2)
    ia, ib = (r0 + 2 * at, r0 + 2 * at + 1) if case["inter"] else (r0 + at, r0 + r // 2 + at)
    turn = np.exp(sign * 1j * pos[:, None, None] * inv_freq[None, None, :])
    w = (v[..., ia] + 1j * v[..., ib]) * turn
    v = v.copy()
    v[..., ia], v[..., ib] = w.real, w.imag
    return v


def _exact_norm_rope(case, s):
    f64 = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    x, pos, f = f64(s["x"]), f64(s["positions"]), f64(s["inv_freq"])
    nd = case["norm_dim"]
    if nd:
        mean = x[..., :nd].mean(-1, keepdims=True) if case["norm"] == "layer" else 0.0
        dev = np.sqrt(((x[..., :nd] - mean) ** 2).mean(-1, keepdims=True) + 1e-6)
        hat, w = (x[..., :nd] - mean) / dev, f64(s["weight"])
    if case["op"] == "fwd":
        y = x.copy()
        if nd:
            y[..., :nd] = hat * w + (f64(s["bias"]) if s["bias"] is not None else 0.0)
        y = _rotated64(case, y, pos, f, 1)
        if not case["slots"]:
            return torch.from_numpy(y)
        full, rows = f64(s["cache"]), s["rows"].cpu().numpy()
        for t, row in enumerate(rows):
            if row >= 0:
                full[row] = y[t]
        return torch.from_numpy(full)
    g = _rotated64(case, f64(s["dout"]), pos, f, -1)
    if not nd:
        return torch.from_numpy(g), None, None
    gy = g[..., :nd]
    dw, db = np.einsum("thd,thd->d", gy, hat), gy.sum((0, 1)) if s["bias"] is not None else None
    # the Jacobian of the normalisation is symmetric: (I - [1 1'/n] - hat hat'/n) / dev
    gw = gy * w
    d = gw - hat * np.einsum("thd,thd->th", gw, hat)[..., None] / nd
    if case["norm"] == "layer":
        d = d - gw.mean(-1, keepdims=True)
    g[..., :nd] = d / dev
    return torch.from_numpy(g), torch.from_numpy(dw), None if db is None else torch.from_numpy(db)


def _exact_mla(case, s):
    b, nq, h, d, k, page = (case[x] for x in ("B", "nq", "H", "D", "K", "page"))
    lens, table = s["seq_lens"].tolist(), s["table"].tolist()
    outs, lses = [], []
    for r in range(b):
        for j in range(nq):
            n = r * nq + j
            v = lens[r] - nq + j + 1
            at = [i for i in s["topk_idx"][n].tolist() if i >= 0] if k else list(range(max(0, v)))
            rows = torch.tensor([table[r][i // page] * page + i % page for i in at], dtype=torch.long, device=DEV)
            kv = s["cache"].reshape(-1, d)[rows].double()
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
    if op in ("slots", "topk"):
        return None  # whole numbers
    if op in ("fwd", "bwd"):
        if case["T"] * case["H"] * case["D"] > 1 << 25:
            return None
        return _exact_norm_rope(case, prepare(case, seed))
    if sum(_lens(case["B"], case["L"])) * case["nq"] * case["H"] > 1 << 27 or case["B"] * case["nq"] > 512:
        return None
    return _exact_mla(case, prepare(case, seed))
