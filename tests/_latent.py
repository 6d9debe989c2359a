"""The latent cache's append and attentions from their definitions, in 64 bits, and seeded inputs for them.

Plain loops over sequences and queries on torch doubles; shares no code with the kernels."""
import math

import torch

D, DV, DR = 576, 512, 64
E4M3 = torch.float8_e4m3fn


def codes_to_double(codes):
    return codes.view(E4M3).double()


def e4m3_round(v):
    """Doubles -> the nearest e4m3 value (ties to even), saturated at 448; NaN for NaN and infinities."""
    a = v.abs().clamp(max=448.0)
    _, e = torch.frexp(a)                                   # a = m 2^e, m in [1/2, 1)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)   # 3 fraction bits, subnormal step 2^-9
    r = torch.round(a / step) * step                        # round half to even
    return torch.where(torch.isfinite(v), torch.copysign(r.clamp(max=448.0), v), math.nan)


def needed_scale(amax):
    e = -40
    while e < 40 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(pe, pos, inv_freq, interleaved):
    """pe double [n, 64], pos list, inv_freq fp32 [32] -> rotated double [n, 64]."""
    th = torch.tensor(pos, dtype=torch.float64, device=pe.device)[:, None] * inv_freq.double()[None]
    i = torch.arange(0, DR, 2, device=pe.device) if interleaved else torch.arange(DR // 2, device=pe.device)
    k = i + 1 if interleaved else i + DR // 2
    out = pe.clone()
    out[:, i] = pe[:, i] * th.cos() - pe[:, k] * th.sin()
    out[:, k] = pe[:, k] * th.cos() + pe[:, i] * th.sin()
    return out


def append_reference(kv, k_pe, inv_freq, interleaved, pool, scales, page_table, q_offsets, q_vis):
    """The cache after the append, as doubles before their rounding to the cache's type: (values, scales,
    written).  Values of an e4m3 cache are in units of their block's scale; written marks the rows whose
    values were set or rescaled, the others hold what they held."""
    ps = pool.shape[1]
    values = (codes_to_double(pool) if scales is not None else pool.double()).reshape(-1, D)
    written = torch.zeros(values.shape[0], dtype=torch.bool, device=pool.device)
    sc = scales.double().reshape(-1).clone() if scales is not None else None
    block = ps // scales.shape[1] if scales is not None else 1
    off, vis = q_offsets.tolist(), q_vis.tolist()
    for b in range(len(off) - 1):
        f = off[b]
        rows = [t for t in range(f, off[b + 1]) if vis[t] > 0]
        if not rows:
            continue
        pos = [vis[t] - 1 for t in rows]
        x = torch.cat([kv[rows].double(), rotate(k_pe[rows].double(), pos, inv_freq, interleaved)], 1)
        slot = [int(page_table[b, p // ps]) * ps + p % ps for p in pos]
        if scales is None:
            values[slot] = x
            written[slot] = True
            continue
        for blk in sorted(set(s // block for s in slot)):
            mine = [i for i, s in enumerate(slot) if s // block == blk]
            first = (vis[f] - 1) + (rows[mine[0]] - f)
            held = (vis[f] - 1) % block if first // block == (vis[f] - 1) // block else 0
            v = x[mine]
            v = v[torch.isfinite(v)]
            s = needed_scale(float(v.abs().max()) if v.numel() else 0.0)
            if held:
                s = max(s, float(sc[blk]))
                if s > float(sc[blk]):
                    old = slice(blk * block, blk * block + held)
                    values[old] = values[old] * (float(sc[blk]) / s)
                    written[old] = True
            sc[blk] = s
            for i in mine:
                values[slot[i]] = x[i] / s
                written[slot[i]] = True
    return values, sc, written


def list_of(vis, sinks, window):
    return [s for s in range(vis) if s < sinks or s >= vis - window]


def attend_reference(q, pool, scales, page_table, q_offsets, lists, scale):
    """(O, LSE, A, z error unit, code floor) over each query's list of positions, in doubles.  A is the sum of
    weight x |value|; the last two are what the tolerances below are made of."""
    ps = pool.shape[1]
    Q, H = q.shape[0], q.shape[1]
    dev = q.device
    out = torch.zeros(Q, H, DV, dtype=torch.float64, device=dev)
    lse = torch.full((Q, H), -math.inf, dtype=torch.float64, device=dev)
    absum = torch.zeros_like(out)
    zunit = torch.zeros(Q, H, dtype=torch.float64, device=dev)
    floor = torch.zeros(Q, DV, dtype=torch.float64, device=dev)
    off = q_offsets.tolist()
    for b in range(len(off) - 1):
        for t in range(off[b], off[b + 1]):
            p = torch.tensor(lists[t], dtype=torch.long, device=dev)
            if not p.numel():
                continue
            pg = page_table[b][p // ps].long()
            row = pool[pg, p % ps]
            if scales is not None:
                s = scales[pg, p % ps // (ps // scales.shape[1])].double()
                code = codes_to_double(row)
                kv = code * s[:, None]
                floor[t] = code[:, :DV].abs().sum(0) * s.max()
            else:
                kv = row.double()
            qd = q[t].double()
            z = qd @ kv.T * scale
            lse[t] = torch.logsumexp(z, 1)
            w = torch.exp(z - lse[t][:, None])
            out[t] = w @ kv[:, :DV]
            absum[t] = w @ kv[:, :DV].abs()
            zunit[t] = (qd.abs() @ kv.abs().T * scale).amax(1)
    return out, lse, absum, zunit, floor


def check_attend(out, lse, ref, e4m3):
    """The kernel's results against attend_reference, element by element.

    A score is 36 accumulation steps of exact 16-bit products, each step off by at most 2^-23 of the sum of
    magnitudes so far, and a few fp32 roundings of its scaling: 40 steps of 2^-23 of zunit.  A weight takes that
    as a relative error, and so does the LSE.  Weights are rounded by at most half a step, 2^-8 (bf16) or 2^-11
    (fp16) relative, with fp16's subnormal half step 2^-25 below (P of the largest weight is at least 1); exp2, the sum
    and the split merge add fp32 roundings, within another 2^-18.  The output is rounded to bf16: 2^-8."""
    o, l, absum, zunit, floor = ref
    empty = torch.isinf(l) & (l < 0)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert (out[empty] == 0).all()
    dz = 40 * 2.0 ** -23 * zunit
    tol_l = torch.where(empty, 0.0, dz + 2.0 ** -18 + 2.0 ** -21 * torch.where(empty, 0.0, l).abs())
    dl = torch.where(empty, 0.0, (lse.double() - l).abs())
    assert (dl <= tol_l).all(), float((dl - tol_l).max())
    weight = (2.0 ** -11 if e4m3 else 2.0 ** -8) + 2.0 ** -18
    tol = 2.0 ** -8 * o.abs() + (1 + 2.0 ** -7) * ((weight + 2 * dz)[..., None] * absum
                                                   + (2.0 ** -25 * floor[:, None, :] if e4m3 else 0.0)) + 1e-30
    do = (out.double() - o).abs()
    assert (do <= tol).all(), float((do / tol).max())


class Cache:
    """A paged cache of seeded values; pages of each sequence are scattered, what no sequence holds is NaN."""

    def __init__(self, lens, page, e4m3, block=1, seed=0, device="cuda", spare=2, scale_exp=(-8, -5)):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.g, self.device, self.page, self.block, self.e4m3 = g, device, page, block, e4m3
        pages = [-(-n // page) for n in lens]
        self.num_pages = sum(pages) + 2
        self.max_pages = max(max(pages), 1) + spare
        perm = torch.randperm(self.num_pages, device=device, generator=g).tolist()
        self.table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32, device=device)
        live = torch.zeros(self.num_pages * page, dtype=torch.bool, device=device)
        at = 0
        for b, n in enumerate(lens):
            mine = perm[at:at + pages[b]]
            at += pages[b]
            if mine:
                self.table[b, :pages[b]] = torch.tensor(mine, dtype=torch.int32, device=device)
                for i, pg in enumerate(mine):
                    live[pg * page:pg * page + min(page, n - i * page)] = True
        x = torch.randn(self.num_pages * page, D, device=device, generator=g)
        if e4m3:
            v = (x * 120).clamp(-448, 448).to(E4M3).view(torch.uint8)
            v[~live] = 0x7F
            self.scales = torch.exp2(torch.randint(scale_exp[0], scale_exp[1] + 1, (self.num_pages, page // block),
                                                   device=device, generator=g).float())
        else:
            v = x.to(torch.bfloat16)
            v[~live] = math.nan
            self.scales = None
        self.pool = v.view(self.num_pages, page, D).contiguous()

    def offsets(self, counts):
        return torch.tensor([0] + counts, device=self.device).cumsum(0).to(torch.int32)
