"""Attention calls whose first query rows lie before the first sequence: the search for a row's sequence stays inside
q_offsets, and the rows of the sequences are what they are without the others."""
import math

import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa
from tests._latent import D, DV, Cache

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5


@pytest.mark.parametrize("B", [1, 2, 33, 70])
@pytest.mark.parametrize("call", ["selected", "sinks", "block"])
def test_rows_before_the_first_sequence(B, call):
    lens = [100 + 3 * b for b in range(B)]
    cache = Cache(lens, 64, call == "block", 64, seed=B)
    before = 3
    Q = before + B
    q = torch.randn(Q, 128, D, device=DEV, generator=cache.g).to(torch.bfloat16)
    vis = torch.tensor([50] * before + lens, dtype=torch.int32, device=DEV)
    idx = torch.stack([torch.randperm(50, device=DEV, generator=cache.g)[:40] for _ in range(Q)]).int().contiguous()
    results = []
    for first in (before, 0):
        n, r = (Q, slice(None)) if first else (B, slice(before, None))
        off = torch.arange(first, first + B + 1, dtype=torch.int32, device=DEV)
        fp32 = call == "selected"
        out = torch.full((n, 128, DV), math.nan, dtype=torch.float32 if fp32 else torch.bfloat16, device=DEV)
        lse = torch.full((n, 128), math.nan, device=DEV)
        args = (q[r].contiguous(), cache.pool, cache.table, off, vis[r].contiguous())
        if call == "selected":
            ws = dsa.workspace(n, 1, 40, 1)
            dsa.dsa_sparse_mla_decode(*args, idx[r].contiguous(), B, SCALE, out, lse, ws, num_splits=1)
        elif call == "sinks":
            ws = dsa.attend_workspace(128)
            dsa.dsa_mla_decode_sinks(*args, B, 4, 60, SCALE, out, lse, ws)
        else:
            ws = dsa.attend_workspace(128)
            dsa.dsa_sparse_mla_decode_fp8_block(args[0], cache.pool, cache.scales, *args[2:], idx[r].contiguous(), B, SCALE, out,
                                                lse, ws)
        dsa.dsa_check_error(ws)
        results.append((out[-B:], lse[-B:]))
    assert not torch.isnan(results[0][0]).any()
    # a query's tiles may be divided otherwise beside other rows: equal up to the parts' merge and the output's rounding
    step = 2.0 ** -8 if call != "selected" else 2.0 ** -10
    scale = results[1][0].float().abs().amax(2, keepdim=True)
    assert ((results[0][0].float() - results[1][0].float()).abs() <= 2 * step * scale).all()
    assert ((results[0][1] - results[1][1]).abs() <= 2.0 ** -10).all()
