"""Operators around the latent cache of an MLA decode step, measured as a serving program calls them.

  append   new tokens' latents go into the paged cache, their position part rotated on the way, as bf16
           or as e4m3 codes with one power-of-two scale for each block of tokens
  sinks    attention of a query over a few first tokens and a sliding window of the last ones, over
           either cache (a window as long as the context is dense attention)
  sparse   attention over the tokens that an indexer selected, over the block-scaled e4m3 cache

The latent row is 512 latent dims and 64 position dims, shared by 64 or 128 query heads.
"""
import math

import torch

own = False

DEV = "cuda"
D, DV, DR = 576, 512, 64
SCALE = 192 ** -0.5
E4M3 = torch.float8_e4m3fn
SCALE_EXP = 40          # block scales are 2^-40 .. 2^40


# ------------------------------------------------------------------ cases
def _append(name, B, lo, hi, ctx, kv8, block, page=64, interleaved=False):
    return dict(name=name, op="append", B=B, lo=lo, hi=hi, ctx=ctx, kv8=kv8, block=block, page=page,
                interleaved=interleaved)


def _sinks(name, B, T, heads, lo, hi, sinks, window, kv8, block, page=64):
    return dict(name=name, op="sinks", B=B, T=T, heads=heads, lo=lo, hi=hi, sinks=sinks, window=window,
                kv8=kv8, block=block, page=page)


def _sparse(name, B, T, heads, lo, hi, topk, block, page=64):
    return dict(name=name, op="sparse", B=B, T=T, heads=heads, lo=lo, hi=hi, topk=topk, kv8=True,
                block=block, page=page)


def listed():
    return [
        # one user's decode step: a single token into a half filled block
        _append("append_b1_fp8", 1, 1, 1, 8191, True, 64),
        # a verify step of 64 users with 1 to 4 new tokens each
        _append("append_verify_b64_fp8", 64, 1, 4, 16000, True, 16),
        # a prompt chunk of four users, bf16 cache
        _append("append_prompt_b4_bf16", 4, 1500, 2500, 4097, False, 64),
        # the largest prompt chunk, block-scaled cache
        _append("append_prompt_b8_fp8", 8, 3000, 5000, 1000, True, 64, interleaved=True),
        # one user, short window, small pages: latency
        _sinks("sinks_b1_h64_bf16_w512", 1, 1, 64, 700, 700, 4, 512, False, 16, page=16),
        # a batch of users past their window
        _sinks("sinks_b32_h128_fp8_w4096", 32, 1, 128, 2000, 16384, 4, 4096, True, 64),
        # dense attention over long contexts: the largest
        _sinks("sinks_full_b4_128k_fp8", 4, 1, 128, 131072, 131072, 0, 131072, True, 64),
        # a verify step of four positions, half the heads
        _sinks("sinks_verify_b24_t4_h64_bf16", 24, 4, 64, 300, 9001, 16, 1024, False, 16),
        # ragged users over the bf16 cache, wide window
        _sinks("sinks_b16_h128_bf16_w8192", 16, 1, 128, 1000, 20001, 4, 8192, False, 64),
        # one user's selected tokens: latency
        _sparse("sparse_b1_fp8", 1, 1, 128, 8192, 8192, 2048, 64),
        # the batch decode of the indexer's selections
        _sparse("sparse_b32_fp8", 32, 1, 128, 32768, 32768, 2048, 64),
        # a verify step of eight positions, half the heads, an odd selection count
        _sparse("sparse_verify_b16_t8_h64_fp8", 16, 8, 64, 700, 16001, 1000, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "sinks", "sparse"])
    page = rng.choice([16, 64])
    block = rng.choice([1, 16, page])
    if op == "append":
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, min(5000, 32768 // B)))
        c = _append(None, B, max(1, hi // rng.choice([1, 2, 5])), hi, _log(rng, 1, 16384), rng.random() < 0.7,
                    block, page, rng.random() < 0.5)
    elif op == "sinks":
        T = rng.choice([1, 1, 2, 4])
        B = _log(rng, 1, 64)
        window = _log(rng, 64, 16384)
        sinks = rng.choice([0, 4, 17, 64])
        hi = _log(rng, 64, min(131072, 262144 // B))
        while B * T * min(hi, sinks + window) > 262144:
            window = window // 2 + 1
        c = _sinks(None, B, T, rng.choice([64, 128]), max(T, hi // rng.choice([1, 3])), hi, sinks, window,
                   rng.random() < 0.6, block, page)
    else:
        T = rng.choice([1, 1, 2, 8])
        B = _log(rng, 1, 64)
        topk = min(_log(rng, 64, 2048), 262144 // (B * T))
        hi = _log(rng, 64, min(131072, 262144 // B))
        c = _sparse(None, B, T, rng.choice([64, 128]), max(T, hi // rng.choice([1, 4])), hi, topk, block, page)
    del c["name"]
    return c


def _spread(lo, hi, B):
    """B lengths between lo and hi, by the case alone."""
    return [lo + int((hi - lo + 1) * ((0.5 + 0.6180339887 * b) % 1.0)) for b in range(B)]


def _lens(c):
    """(tokens visible to each sequence's last query, queries of each sequence)."""
    if c["op"] == "append":
        n = _spread(c["lo"], c["hi"], c["B"])
        old = _spread(0, c["ctx"], c["B"]) if c["B"] > 1 else [c["ctx"]]
        return [o + k for o, k in zip(old, n)], n
    return _spread(c["lo"], c["hi"], c["B"]), [c["T"]] * c["B"]


def work(case):
    c = case
    ctx, n = _lens(c)
    T = sum(n)
    row = D * (1 if c["kv8"] else 2)
    if c["op"] == "append":
        return {"bytes": T * (D * 2 + row) + (8 * T / c["block"] if c["kv8"] else 0), "flops": 6 * DR / 2 * T}
    H = c["heads"]
    rows = pairs = 0
    for L, t in zip(ctx, n):
        if c["op"] == "sparse":
            pairs += sum(min(c["topk"], L - t + 1 + i) for i in range(t))
            rows += min(L, t * c["topk"])
        else:
            pairs += sum(min(L - t + 1 + i, c["sinks"] + c["window"]) for i in range(t))
            rows += min(L, c["sinks"] + c["window"] + t - 1)
    io = T * H * (D * 2 + DV * 2 + 4)
    return {"bytes": rows * row + io + (T * c["topk"] * 4 if c["op"] == "sparse" else 0),
            "flops": 2 * H * (D + DV) * pairs}


# ------------------------------------------------------------------ inputs
def _codes(shape, g):
    return (torch.randn(shape, device=DEV, generator=g) * 120).clamp_(-448, 448).to(E4M3).view(torch.uint8)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    ctx, n = _lens(c)
    B, ps, T = c["B"], c["page"], sum(n)
    pages = [-(-L // ps) for L in ctx]
    max_pages = max(pages) + 1
    num_pages = sum(pages) + 3
    perm = torch.randperm(num_pages, device=DEV, generator=g).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    at = torch.tensor([0] + pages, device=DEV).cumsum(0)
    col = torch.arange(max_pages, device=DEV)
    have = col[None] < torch.tensor(pages, device=DEV)[:, None]
    table[have] = perm[(at[:-1, None] + col[None])[have]]
    q_offsets = torch.tensor([0] + n, device=DEV).cumsum(0).to(torch.int32)
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(n, device=DEV))
    t = torch.arange(T, device=DEV)
    q_vis = (torch.tensor(ctx, device=DEV)[seq] - (q_offsets[1:].long()[seq] - 1 - t)).to(torch.int32)
    s = dict(case=c, B=B, T=T, page_table=table, q_offsets=q_offsets, q_vis=q_vis, max_ctx=max(ctx))
    if c["kv8"]:
        s["pool"] = _codes((num_pages, ps, D), g)
        s["scales"] = torch.exp2(torch.randint(-8, -4, (num_pages, ps // c["block"]), device=DEV, generator=g).float())
    else:
        s["pool"] = torch.randn(num_pages, ps, D, device=DEV, generator=g).to(torch.bfloat16)
        s["scales"] = None
    if c["op"] == "append":
        # the projection's output: latent and position parts of one row
        x = torch.randn(T, D, device=DEV, generator=g) * torch.exp(0.7 * torch.randn(T, 1, device=DEV, generator=g))
        x = x.to(torch.bfloat16)
        s["kv"], s["k_pe"] = x[:, :DV], x[:, DV:]
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, DR, 2, device=DEV, dtype=torch.float64) / DR)).float()
    else:
        s["q"] = torch.randn(T, c["heads"], D, device=DEV, generator=g).to(torch.bfloat16)
        s["out"] = torch.empty(T, c["heads"], DV, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(T, c["heads"], dtype=torch.float32, device=DEV)
    if c["op"] == "sparse":
        K = c["topk"]
        # distinct positions of each query, in no order; -1 behind them where it sees fewer than topk
        L = max(ctx)
        idx = torch.empty(T, K, dtype=torch.int32, device=DEV)
        step = max(1, (1 << 26) // L)
        for r in range(0, T, step):
            v = q_vis[r:r + step, None]
            key = torch.rand(v.shape[0], L, device=DEV, generator=g)
            key.masked_fill_(torch.arange(L, device=DEV)[None] >= v, 2.0)
            k = min(K, L)
            top = key.topk(k, dim=1, largest=False)
            idx[r:r + step, :k] = torch.where(top.values < 1.5, top.indices, -1).to(torch.int32)
            idx[r:r + step, k:] = -1
        s["idx"] = idx
    # the workspace that a program keeps, zeroed once: the error word, and room for partial results
    s["ws"] = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ the plain forms
def _pow2_scale(amax):
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875)
    e = torch.where(amax > 0, e, -SCALE_EXP).clamp(-SCALE_EXP, SCALE_EXP)
    return torch.exp2(e.float())


def _e4m3(x):
    return torch.where(torch.isfinite(x), x.clamp(-448.0, 448.0), math.nan).to(E4M3)


def _plain_append(s):
    c = s["case"]
    ps, block = c["page"], c["block"]
    seq = torch.searchsorted(s["q_offsets"][1:], torch.arange(s["T"], device=DEV), right=True)
    pos = s["q_vis"].long() - 1
    angle = pos.double()[:, None] * s["inv_freq"].double()[None]
    cos, sin = angle.cos().float(), angle.sin().float()
    pe = s["k_pe"].float()
    if c["interleaved"]:
        a, b = pe[:, 0::2], pe[:, 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=2).flatten(1)
    else:
        a, b = pe[:, :DR // 2], pe[:, DR // 2:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=1)
    x = torch.cat([s["kv"].float(), rot], dim=1)
    slot = s["page_table"][seq, pos // ps].long() * ps + pos % ps
    if not c["kv8"]:
        s["pool"].view(-1, D)[slot] = x.to(torch.bfloat16)
        return s["pool"]
    pool, scales = s["pool"].view(E4M3).view(-1, D), s["scales"].view(-1)
    blk = slot // block
    amax = torch.zeros_like(scales).scatter_reduce(0, blk, x.abs().amax(1), "amax")
    new = _pow2_scale(amax)
    # each sequence's first block may hold tokens already: its scale never falls, and they are scaled with it
    f = s["q_offsets"][:-1].long()
    held = slot[f] % block
    b0 = blk[f]
    old = scales[b0]
    new[b0] = torch.where(held > 0, torch.maximum(old, new[b0]), new[b0])
    ratio = old / new[b0]
    rows = b0[:, None] * block + torch.arange(block, device=DEV)[None]
    codes = pool.view(torch.uint8)[rows]
    again = _e4m3(codes.view(E4M3).float() * ratio[:, None, None]).view(torch.uint8)
    keep = torch.arange(block, device=DEV)[None, :, None] >= held[:, None, None]
    pool.view(torch.uint8)[rows] = torch.where(keep, codes, again)
    scales[blk] = new[blk]
    pool.view(torch.uint8)[slot] = _e4m3(x / new[blk][:, None]).view(torch.uint8)
    return s["pool"].view(E4M3), s["scales"]


def _plain_attend(s):
    c = s["case"]
    ps = c["page"]
    vis = s["q_vis"].long()[:, None]
    if c["op"] == "sparse":
        pos = s["idx"].long()
        ok = pos >= 0
    else:
        n = min(s["max_ctx"], c["sinks"] + c["window"])
        j = torch.arange(n, device=DEV)[None]
        ns = vis.clamp(max=c["sinks"])
        w0 = torch.maximum(ns, vis - c["window"])
        pos = torch.where(j < ns, j, w0 + j - ns)
        ok = pos < vis
    pos = torch.where(ok, pos, 0)
    seq = torch.searchsorted(s["q_offsets"][1:], torch.arange(s["T"], device=DEV), right=True)
    page = s["page_table"][seq[:, None], pos // ps].long()
    kv = s["pool"].view(E4M3).view(-1, D) if c["kv8"] else s["pool"].view(-1, D)
    kv = (kv.view(torch.uint8) if c["kv8"] else kv)[page * ps + pos % ps]
    kv = kv.view(E4M3).float() if c["kv8"] else kv.float()
    if c["kv8"]:
        kv *= s["scales"][page, pos % ps // c["block"]][:, :, None]
    kv.masked_fill_(~ok[:, :, None], 0.0)
    z = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * SCALE
    z.masked_fill_(~ok[:, None, :], -math.inf)
    m = z.amax(2, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(z - m)
    l = p.sum(2, keepdim=True)
    o = torch.matmul(p, kv[:, :, :DV]) / l.clamp(min=1e-38)
    return o.to(torch.bfloat16), (m + torch.log(l)).squeeze(2)


# ------------------------------------------------------------------ the calls
def run(state):
    s = state
    c = s["case"]
    if not own:
        return _plain_append(s) if c["op"] == "append" else _plain_attend(s)
    import sparse_attention_decode_lightning_b200 as dsa
    if c["op"] == "append":
        dsa.dsa_latent_append(s["kv"], s["k_pe"], s["inv_freq"], s["pool"], s["page_table"], s["q_offsets"],
                              s["q_vis"], s["B"], s["ws"], kv_scales=s["scales"], interleaved=c["interleaved"])
        return (s["pool"].view(E4M3), s["scales"]) if c["kv8"] else s["pool"]
    if c["op"] == "sinks":
        dsa.dsa_mla_decode_sinks(s["q"], s["pool"], s["page_table"], s["q_offsets"], s["q_vis"], s["B"], c["sinks"],
                                 c["window"], SCALE, s["out"], s["lse"], s["ws"], kv_scales=s["scales"])
    else:
        dsa.dsa_sparse_mla_decode_fp8_block(s["q"], s["pool"], s["scales"], s["page_table"], s["q_offsets"],
                                            s["q_vis"], s["idx"], s["B"], SCALE, s["out"], s["lse"], s["ws"])
    return s["out"], s["lse"]


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_append(s):
    c = s["case"]
    ps, block = c["page"], c["block"]
    off = s["q_offsets"].tolist()
    vis = s["q_vis"].tolist()
    table = s["page_table"].tolist()
    x = torch.cat([s["kv"], s["k_pe"]], 1).double()
    freq = s["inv_freq"].double()
    pool = (s["pool"].view(E4M3) if c["kv8"] else s["pool"]).double().view(-1, D)
    scales = s["scales"].double().view(-1) if c["kv8"] else None
    i, k = (torch.arange(0, DR, 2, device=DEV), torch.arange(1, DR, 2, device=DEV)) if c["interleaved"] else (
        torch.arange(DR // 2, device=DEV), torch.arange(DR // 2, DR, device=DEV))
    for b in range(s["B"]):
        t0, t1 = off[b], off[b + 1]
        p0 = vis[t0] - 1
        th = (p0 + torch.arange(t1 - t0, device=DEV, dtype=torch.float64))[:, None] * freq
        y = x[t0:t1].clone()
        u, w = x[t0:t1, DV + i], x[t0:t1, DV + k]
        y[:, DV + i] = u * torch.cos(th) - w * torch.sin(th)
        y[:, DV + k] = w * torch.cos(th) + u * torch.sin(th)
        if not c["kv8"]:
            p = p0 + torch.arange(t1 - t0, device=DEV)
            tab = torch.tensor(table[b], device=DEV)
            pool[tab[p // ps] * ps + p % ps] = y
            continue
        top = y.abs().amax(1).tolist()
        t = 0
        while t < t1 - t0:                      # one block of tokens at a time
            p = p0 + t
            n = min(block - p % block, t1 - t0 - t)
            row = table[b][p // ps] * ps + p % ps
            a = max(top[t:t + n])
            e = -SCALE_EXP if a == 0 else max(-SCALE_EXP, min(SCALE_EXP, math.ceil(math.log2(a / 448.0) - 1e-15)))
            sc = 2.0 ** e
            held = p % block
            at = row // block
            if held:
                was = float(scales[at])
                sc = max(sc, was)
                if sc != was:
                    pool[row - held:row] *= was / sc
            scales[at] = sc
            pool[row:row + n] = y[t:t + n] / sc
            t += n
    shape = s["pool"].shape
    return pool.view(shape) if not c["kv8"] else (pool.view(shape), scales.view(s["scales"].shape))


def _exact_attend(s):
    c = s["case"]
    ps = c["page"]
    off, vis = s["q_offsets"].tolist(), s["q_vis"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b in range(s["B"]):
        for t in range(off[b], off[b + 1]):
            v = vis[t]
            if c["op"] == "sparse":
                p = s["idx"][t][s["idx"][t] >= 0].long()
            else:
                p = torch.arange(v, device=DEV)
                p = p[(p < c["sinks"]) | (p >= v - c["window"])]
            if not p.numel():
                continue
            pg = s["page_table"][b][p // ps].long()
            kv = s["pool"][pg, p % ps]
            kv = kv.view(E4M3).double() * s["scales"][pg, p % ps // c["block"]].double()[:, None] if c["kv8"] else kv.double()
            z = (s["q"][t].double() @ kv.T) / math.sqrt(192.0)
            lse[t] = torch.logsumexp(z, 1)
            out[t] = torch.exp(z - lse[t][:, None]) @ kv[:, :DV]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
