"""The block-scaled attentions where tokens of one tile have scales far apart and the small ones carry the output: every
token that weighs enough has to reach it, whatever scale its neighbours have."""
import math

import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa
from tests._latent import D, DV, E4M3, Cache, attend_reference, codes_to_double

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5
PEAK = 0.875                                     # place of the heaviest token along the list
Z = DV + 63                                      # the dim that carries the scores: a position dim, no value


def codes(v):
    return v.clamp(-448, 448).to(E4M3).view(torch.uint8)


def make(n, ratio, mass, heads, outliers, values):
    """A cache with a scale a token.  One token weighs 1; the others, of the same scale 1, `mass` together; in each tile
    of 128 tokens (or in the heaviest one's alone) one token has the scale 2^ratio, and a score so low that its product
    of weight and scale is below 2^-45."""
    cache = Cache([n], 64, True, 1, seed=n + ratio)
    pos = torch.arange(n, device=DEV)
    slot = cache.table[0].long()[pos // 64] * 64 + pos % 64
    flat, scales = cache.pool.view(-1, D), cache.scales.view(-1)
    scales[slot] = 1.0
    v = 64 * (0.5 + torch.rand(n, D, device=DEV, generator=cache.g))
    peak = int(PEAK * n)
    v[peak] = 0 if values == "none" else 64 * torch.randn(D, device=DEV, generator=cache.g)
    gap = math.log2(n / mass)                    # of the heaviest score above the others, in bits
    v[:, Z] = 0
    v[peak, Z] = 448
    out = pos[(pos % 128 == 5) & ((pos // 128 == peak // 128) | (outliers == "all"))]
    # at least 2^-9, e4m3's smallest: the score is then below -(50 + ratio) bits all the same
    v[out, Z] = -max(448 * (50 + ratio) / (gap * 2.0 ** ratio), 2.0 ** -9)
    flat[slot] = codes(v)
    scales[slot[out]] = 2.0 ** ratio
    q = torch.zeros(1, heads, D, device=DEV)
    q[0, :, Z] = gap * math.log(2) / (SCALE * 448) * torch.linspace(0.92, 1.0, heads, device=DEV)
    return cache, q.to(torch.bfloat16)


def check(cache, q, out, lse, positions):
    """Element by element.  A score is one exact product and zeros, so its error is the fp32 roundings of its scaling
    by the token's scale, the query's factor and log2 of the scale and of the difference to the maximum: four of 2^-24
    of the largest magnitude in bits.  A weight takes that, times ln 2 < 1, twice (numerator and sum); it is rounded
    to fp16 by 2^-11 of itself where weight x scale is at least 2^-21 of the largest such product, and may be lost
    whole below.  Values are summed 16 tokens a step over the tiles that one pair of SMs takes, each step off by at most
    2^-23 of the sum; exp2, the weights' sum and the merge of parts are within another 2^-18.  The output is rounded to
    bf16: 2^-8."""
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    o, l, absum, _, _ = attend_reference(q, cache.pool, cache.scales, cache.table, off, [positions], SCALE)
    p = torch.tensor(positions, device=DEV)
    page = cache.table[0].long()[p // 64]
    s = cache.scales[page, p % 64].double()
    kv = codes_to_double(cache.pool[page, p % 64]) * s[:, None]
    z = q[0].double() @ kv.T * SCALE
    w = torch.exp(z - l[0][:, None])
    small = w * s < 2.0 ** -21 * (w * s).amax(1, keepdim=True)
    lost = torch.where(small, w, 0.0) @ kv[:, :DV].abs()
    # what the small ones contribute is next to nothing: the bound below says something
    assert (lost <= 2.0 ** -12 * absum[0]).all()
    dz = 4 * 2.0 ** -24 * ((z.abs().amax(1) + l[0].abs()) / math.log(2) + 2 * torch.log2(s).abs().max())
    steps = 8 * (len(positions) // (128 * 74) + 1)
    tol = 2.0 ** -8 * o[0].abs() + (1 + 2.0 ** -7) * ((2.0 ** -11 + 2.0 ** -18 + steps * 2.0 ** -23 + 2 * dz)[:, None] * absum[0] + lost)
    err = (out[0].double() - o[0]).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert ((lse[0].double() - l[0]).abs() <= dz + 2.0 ** -18).all()


# tokens, log2 of the outliers' scale, weight of all tokens but the heaviest over its own
CASES = [(131072, 5, 0.11), (131072, 8, 0.84), (131072, 11, 0.84), (16384, 10, 1.6), (16384, 15, 8.0), (4096, 14, 1.42),
         (4096, 2, 0.01)]


@pytest.mark.parametrize("n,ratio,mass", CASES)
@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("outliers", ["all", "one"])
@pytest.mark.parametrize("values", ["some", "none"])
def test_a_long_tail_beside_one_large_scale(n, ratio, mass, heads, outliers, values):
    cache, q = make(n, ratio, mass, heads, outliers, values)
    out = torch.full((1, heads, DV), math.nan, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((1, heads), math.nan, device=DEV)
    ws = dsa.attend_workspace(heads)
    off, vis = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([0, 1], [n]))
    dsa.dsa_mla_decode_sinks(q, cache.pool, cache.table, off, vis, 1, 0, n, SCALE, out, lse, ws, kv_scales=cache.scales)
    dsa.dsa_check_error(ws)
    check(cache, q, out, lse, list(range(n)))


@pytest.mark.parametrize("ratio,mass", [(5, 0.1), (11, 0.84), (14, 1.42)])
@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("values", ["some", "none"])
def test_selected_tokens_beside_one_large_scale(ratio, mass, heads, values):
    n = 2048
    cache, q = make(n, ratio, mass, heads, "all", values)
    pick = torch.randperm(n, device=DEV, generator=cache.g)
    out = torch.full((1, heads, DV), math.nan, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((1, heads), math.nan, device=DEV)
    ws = dsa.attend_workspace(heads)
    off, vis = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([0, 1], [n]))
    dsa.dsa_sparse_mla_decode_fp8_block(q, cache.pool, cache.scales, cache.table, off, vis, pick.to(torch.int32)[None].contiguous(),
                                        1, SCALE, out, lse, ws)
    dsa.dsa_check_error(ws)
    check(cache, q, out, lse, pick.tolist())
