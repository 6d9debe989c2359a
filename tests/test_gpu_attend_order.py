"""Attention enqueued directly behind what writes its inputs: it starts beside that kernel's end and must see all of it."""
import math

import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa
from tests._latent import D, DV, Cache

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5
STEPS = 24


def decode(selected, wait):
    """Steps of two users: copies rewrite the page table, offsets and q_vis; the append writes codes and scales (each
    step's tokens are larger or smaller by powers of two); the attention follows at once, or after the GPU is idle."""
    cache = Cache([400, 300], 64, True, 64, seed=7)
    g = cache.g
    ws = dsa.attend_workspace(128)
    freq = torch.rand(32, device=DEV, generator=g)
    tables = [cache.table.clone(), cache.table.flip(1).flip(1).clone()]
    tables[1][:, [0, 1]] = tables[1][:, [1, 0]]
    x = [(torch.randn(128, D, device=DEV, generator=g) * 2.0 ** (i % 7)).to(torch.bfloat16) for i in range(STEPS)]
    q = [torch.randn(2, 128, D, device=DEV, generator=g).to(torch.bfloat16) for _ in range(STEPS)]
    idx = [torch.stack([torch.randperm(250, device=DEV, generator=g)[:200] for _ in range(2)]).int() for _ in range(STEPS)]
    append_off = torch.tensor([0, 64, 128], dtype=torch.int32, device=DEV)
    append_vis = torch.cat([torch.arange(192, 256), torch.arange(64, 128)]).int().to(DEV) + 1
    off = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    vis = torch.zeros(2, dtype=torch.int32, device=DEV)
    table, at, mine = cache.table.clone(), torch.zeros(2, 200, dtype=torch.int32, device=DEV), torch.empty_like(q[0])
    results = []
    torch.cuda.synchronize()
    for i in range(STEPS):
        table.copy_(tables[i % 2])
        at.copy_(idx[i])
        mine.copy_(q[i])
        vis.fill_(260 + i % 5)
        dsa.dsa_latent_append(x[i][:, :DV], x[i][:, DV:], freq, cache.pool, table, append_off, append_vis, 2, ws,
                              kv_scales=cache.scales)
        if wait:
            torch.cuda.synchronize()
        out = torch.full((2, 128, DV), math.nan, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((2, 128), math.nan, device=DEV)
        if wait:
            torch.cuda.synchronize()
        if selected:
            dsa.dsa_sparse_mla_decode_fp8_block(mine, cache.pool, cache.scales, table, off, vis, at, 2, SCALE, out, lse, ws)
        else:
            dsa.dsa_mla_decode_sinks(mine, cache.pool, table, off, vis, 2, 0, 1 << 30, SCALE, out, lse, ws,
                                     kv_scales=cache.scales)
        results.append((out, lse))
        if wait:
            torch.cuda.synchronize()
    dsa.dsa_check_error(ws)
    return results


@pytest.mark.parametrize("selected", [False, True])
def test_attention_right_behind_the_writers_of_its_inputs(selected):
    for (a, b), (c, d) in zip(decode(selected, False), decode(selected, True)):
        assert not torch.isnan(a).any()
        assert torch.equal(a, c) and torch.equal(b, d)
