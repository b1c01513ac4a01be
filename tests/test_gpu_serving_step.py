"""A few decode steps of a small sparse-attention layer through the paged calls, one after the other as a serving loop
makes them, captured into one graph and replayed while the requests grow: the slots of the new tokens, their latents and
index keys (norm and rotation) into the caches, the rotation of the queries in place, the selection, the attention over
it; against a request-by-request computation in 64 bits that keeps its own caches."""
import numpy as np
import pytest
import torch

import sparse_attention_mla_gb300 as dsa

import _paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def f64(t):
    return t.detach().cpu().double().numpy()


def test_decode_steps():
    B, H, Hi, P, K, steps = 3, 16, 8, 16, 40, 5
    start, pages = [70, 0, 31], 24
    g = torch.Generator().manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    freq, rscale = dsa.dsa_rope_frequencies(64, factor=4.0, original_context=64)
    lat_w, key_w, key_b = 1 + 0.1 * rand(512), 1 + 0.1 * rand(128), 0.1 * rand(128)
    # prompts: latents and keys already in their pages
    table = torch.full((B, 8), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).tolist()
    for b, n in enumerate(start):
        for c in range(-(-n // P)):
            table[b, c] = order.pop()
    kv, keys = rand(pages, P, 576).bfloat16(), rand(pages, P, 128).bfloat16()
    d = lambda t: t.to(DEV)  # noqa: E731
    cache, kcache, tab, lens = d(kv), d(keys), d(table), d(torch.tensor(start, dtype=torch.int32))
    free = d(torch.tensor(order, dtype=torch.int32))
    x_lat, x_key = torch.empty(B, 576, dtype=torch.bfloat16, device=DEV), torch.empty(B, 128, dtype=torch.bfloat16, device=DEV)
    q, qi = torch.empty(B, H, 576, dtype=torch.bfloat16, device=DEV), torch.empty(B, Hi, 128, dtype=torch.bfloat16, device=DEV)
    w = d(torch.rand(B, Hi, generator=g))
    lw, kw_, kb = d(lat_w), d(key_w), d(key_b)
    scratch = {k: torch.zeros(n, dtype=torch.uint8, device=DEV) for k, n in
               (("a", 256), ("t", dsa.paged_workspace_size("topk", B, 8 * P)), ("m", dsa.paged_workspace_size("mla")))}

    def step():
        slots, pos, cu, new_lens, taken = dsa.dsa_paged_slots(lens, tab, free, P, workspace=scratch["a"])
        dsa.dsa_norm_rope_fwd(x_lat, freq, pos, "rms", 512, lw, rope_scale=rscale, interleaved=True, out=cache,
                              out_rows=slots, workspace=scratch["a"])
        dsa.dsa_norm_rope_fwd(x_key, freq, pos, "layer", 128, kw_, kb, rope_start=0, rope_scale=rscale, out=kcache,
                              out_rows=slots, workspace=scratch["a"])
        qr = q[..., 512:]
        dsa.dsa_norm_rope_fwd(qr, freq, pos, rope_scale=rscale, interleaved=True, out=qr, workspace=scratch["a"])
        dsa.dsa_norm_rope_fwd(qi, freq, pos, rope_start=0, rope_scale=rscale, out=qi, workspace=scratch["a"])
        idx, ln = dsa.dsa_paged_indexer_topk(qi, kcache, w, tab, new_lens, K, workspace=scratch["t"])
        out, lse = dsa.dsa_paged_mla(q, cache, tab, new_lens, 0.05, topk_idx=idx, topk_len=ln, workspace=scratch["m"])
        return new_lens, taken, idx, ln, out, lse

    def inputs(seed):
        gg = torch.Generator().manual_seed(seed)
        v = [torch.randn(*t.shape, generator=gg).bfloat16() for t in (x_lat, x_key, q, qi)]
        for t, s in zip((x_lat, x_key, q, qi), v):
            t.copy_(s)
        return v

    # a warm-up on copies of the state, then the capture
    keep = [t.clone() for t in (cache, kcache, tab)]
    inputs(0)
    step()
    torch.cuda.synchronize()
    for t, s in zip((cache, kcache, tab), keep):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new_lens, taken, idx, ln, out, lse = step()
    f, w64 = f64(freq), w.cpu()
    n, rest = list(start), list(order)
    for k in range(steps):
        lat, key, qs, qis = inputs(100 + k)
        graph.replay()
        for b in range(B):  # the same step on the host
            if n[b] % P == 0:
                table[b, n[b] // P] = rest.pop(0)
            at = ref.rows_of(table[b], [n[b]], P)[0]
            pos = np.array([float(n[b])])
            y = ref.norm_rope_fwd(f64(lat[b:b + 1, None]), "rms", 512, f64(lat_w), None, 1e-6, pos, f, 512, True, rscale)[0, 0]
            z = ref.norm_rope_fwd(f64(key[b:b + 1, None]), "layer", 128, f64(key_w), f64(key_b), 1e-6, pos, f, 0, False, rscale)[0, 0]
            got, got_k = f64(cache.view(-1, 576)[at]), f64(kcache.view(-1, 128)[at])
            assert np.all(np.abs(got - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -13 * np.abs(y).max())
            assert np.all(np.abs(got_k - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -13 * np.abs(z).max())
            kv.view(-1, 576)[at], keys.view(-1, 128)[at] = cache.view(-1, 576)[at].cpu(), kcache.view(-1, 128)[at].cpu()
            n[b] += 1
        assert torch.equal(tab.cpu(), table) and new_lens.tolist() == n
        assert torch.equal(cache.cpu(), kv) and torch.equal(kcache.cpu(), keys)  # no other row was touched
        # the queries as the calls turned them, so that the selections can be compared
        qt, qit = q.cpu(), qi.cpu()
        for b in range(B):
            s, mag = ref.paged_scores(qit[b], keys, w64[b], table[b], n[b], P)
            want = ref.topk_of(s, K)
            sel = idx[b, :int(ln[b])].tolist()
            assert len(sel) == len(want)
            for x in set(sel) ^ set(want):
                kth = min(want, key=lambda i: float(s[i]))
                assert abs(float(s[x] - s[kth])) <= 200 * 2.0 ** -24 * float(mag[x] + mag[kth])
        want_o, want_l = ref.paged_mla(qt, kv, table.tolist(), n, list(range(B + 1)), 0.05, P, topk=idx.cpu(), topk_len=ln.cpu())
        o = out.cpu().double()
        assert bool(((o - want_o).abs() <= 2.0 ** -8 * want_o.abs() + 2.0 ** -13 * 6).all())
        assert bool(((lse.cpu().double() - want_l).abs() <= 2.0 ** -13).all())
        lens.copy_(new_lens)
        free.copy_(torch.roll(free, -int(taken)))
    for t in scratch.values():
        assert dsa.dsa_read_device_status(t) == 0
