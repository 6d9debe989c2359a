"""Calls of the latent cache's operators that the argument lists allow: counts beyond 32 bits, offsets that leave the
rows."""
import math

import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa
from tests._latent import D, DV, Cache

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("sinks,window", [(0, 1 << 32), (0, 1 << 40), (0, (1 << 63) - 1), (1 << 40, 0), (1 << 32, 1 << 32)])
def test_a_count_beyond_32_bits_is_dense_attention(e4m3, sinks, window):
    lens = [700, 1, 129]
    cache = Cache(lens, 64, e4m3, 16, seed=3)
    q = torch.randn(3, 128, D, device=DEV, generator=cache.g).to(torch.bfloat16)
    off, vis = cache.offsets([1] * 3), torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = dsa.attend_workspace(128)
    results = []
    for s, w in ((0, 700), (sinks, window)):
        out = torch.full((3, 128, DV), math.nan, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((3, 128), math.nan, device=DEV)
        dsa.dsa_mla_decode_sinks(q, cache.pool, cache.table, off, vis, 3, s, w, SCALE, out, lse, ws, kv_scales=cache.scales)
        results.append((out, lse))
    dsa.dsa_check_error(ws)
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("offsets", [[0, 3, 9], [-2, 3, 6]])
def test_offsets_that_leave_the_rows_are_flagged(e4m3, offsets):
    """A sequence that ends behind the last row, or begins before the first: not appended, and said so."""
    cache = Cache([40, 40], 16, e4m3, 16, seed=4)
    x = torch.randn(6, D, device=DEV, generator=cache.g).to(torch.bfloat16)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    vis = torch.tensor([1, 2, 3, 1, 2, 3], dtype=torch.int32, device=DEV)
    if offsets[0] < 0:
        vis[:3] += 2                                              # as if two rows lay before
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    before = cache.pool.clone()
    dsa.dsa_latent_append(x[:, :DV], x[:, DV:], torch.ones(32, device=DEV), cache.pool, cache.table, off, vis, 2, ws,
                          kv_scales=cache.scales)
    with pytest.raises(dsa.DSAError) as e:
        dsa.dsa_check_error(ws)
    assert e.value.status == 4
    bits = torch.uint8 if e4m3 else torch.int16
    bad, good = (1, 0) if offsets[0] == 0 else (0, 1)
    page = cache.table[:, 0].long()
    assert torch.equal(cache.pool[page[bad]].view(bits), before[page[bad]].view(bits))
    assert not torch.equal(cache.pool[page[good], :3].view(bits), before[page[good], :3].view(bits))
