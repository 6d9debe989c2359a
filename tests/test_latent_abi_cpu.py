"""Refusals of the latent cache's append and attentions: the host checks of the C ABI (nothing is enqueued, so made-up
pointers do) and the binding's checks of types and shapes."""
import math

import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa
from tests._latent import e4m3_round

OK_PTR, ODD = 1 << 20, (1 << 20) + 4
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_attention_decode_lightning_b200.build import build
    build()


def append(**over):
    a = dict(kv=OK_PTR, ld_kv=576, k_pe=OK_PTR, ld_pe=576, inv_freq=OK_PTR, inter=0, table=OK_PTR, max_pages=4,
             off=OK_PTR, vis=OK_PTR, B=2, T=3, pool=OK_PTR, scales=OK_PTR, num_pages=8, page=64, block=16, ws=OK_PTR,
             ws_bytes=256, stream=None)
    a.update(over)
    return dsa.lib().dsa_latent_append(*a.values())


def sinks(**over):
    a = dict(q=OK_PTR, pool=OK_PTR, scales=OK_PTR, num_pages=8, page=64, block=16, table=OK_PTR, max_pages=4, off=OK_PTR,
             vis=OK_PTR, B=2, Q=3, heads=128, sinks=4, window=100, scale=0.1, out=OK_PTR, lse=OK_PTR, ws=OK_PTR,
             ws_bytes=dsa.dsa_attend_workspace_bytes(128), stream=None)
    a.update(over)
    return dsa.lib().dsa_mla_decode_sinks(*a.values())


def sparse(**over):
    a = dict(q=OK_PTR, pool=OK_PTR, scales=OK_PTR, num_pages=8, page=64, block=16, table=OK_PTR, max_pages=4, off=OK_PTR,
             vis=OK_PTR, idx=OK_PTR, B=2, Q=3, heads=128, topk=64, scale=0.1, out=OK_PTR, lse=OK_PTR, ws=OK_PTR,
             ws_bytes=dsa.dsa_attend_workspace_bytes(128), stream=None)
    a.update(over)
    return dsa.lib().dsa_sparse_mla_decode_fp8_block(*a.values())


CACHE = [
    (dict(pool=None), INVALID), (dict(pool=ODD), INVALID), (dict(table=None), INVALID), (dict(num_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(page=48), UNSUPPORTED), (dict(page=2048), UNSUPPORTED), (dict(page=0), UNSUPPORTED),
    (dict(num_pages=1 << 30), UNSUPPORTED), (dict(block=0), UNSUPPORTED), (dict(block=3), UNSUPPORTED),
    (dict(block=128), UNSUPPORTED), (dict(scales=OK_PTR + 2), INVALID), (dict(off=None), INVALID), (dict(vis=None), INVALID),
    (dict(B=0), INVALID), (dict(B=2049), UNSUPPORTED), (dict(ws=None), INVALID), (dict(ws_bytes=255), WORKSPACE),
]


@pytest.mark.parametrize("over,status", CACHE + [
    (dict(kv=None), INVALID), (dict(k_pe=None), INVALID), (dict(inv_freq=None), INVALID), (dict(T=0), INVALID),
    (dict(kv=ODD), INVALID), (dict(ld_kv=511), INVALID), (dict(ld_kv=577), INVALID), (dict(ld_pe=62), INVALID),
    (dict(ld_pe=65), INVALID), (dict(k_pe=OK_PTR + 2), INVALID)])
def test_append_refuses(over, status):
    assert append(**over) == status


ATTEND = CACHE + [
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(out=None), INVALID), (dict(out=ODD), INVALID),
    (dict(lse=None), INVALID), (dict(ws=ODD), INVALID), (dict(Q=0), INVALID), (dict(Q=65536), UNSUPPORTED),
    (dict(heads=32), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(ws_bytes=dsa.PAGE_SIZE), WORKSPACE)]


@pytest.mark.parametrize("over,status", ATTEND + [(dict(sinks=-1), INVALID), (dict(window=-1), INVALID)])
def test_sinks_refuses(over, status):
    assert sinks(**over) == status


@pytest.mark.parametrize("over,status", ATTEND + [(dict(idx=None), INVALID), (dict(topk=0), INVALID),
                                                  (dict(topk=2049), UNSUPPORTED), (dict(scales=None), INVALID)])
def test_selected_refuses(over, status):
    assert sparse(**over) == status


def test_workspace_bytes():
    f = dsa.dsa_attend_workspace_bytes
    assert f(32) == 0 and f(0) == 0
    # two parts a pair of SMs (74), fp32 output and log-sum-exp, and a header
    assert f(128) >= 2 * 74 * 128 * 513 * 4 and f(64) >= 2 * 74 * 64 * 513 * 4
    assert f(64) < f(128) <= 1 << 26
    with pytest.raises(dsa.DSAError):
        dsa.attend_workspace(96, device="cpu")


def test_binding_refuses_host_tensors_and_wrong_types():
    t = torch.zeros
    kv, pe = t(3, 512, dtype=torch.bfloat16), t(3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.dsa_latent_append(kv, pe, t(32), t(4, 64, 576, dtype=torch.bfloat16), t(1, 4, dtype=torch.int32),
                              t(2, dtype=torch.int32), t(3, dtype=torch.int32), 1, t(256, dtype=torch.uint8))
    q, out, lse = t(2, 128, 576, dtype=torch.bfloat16), t(2, 128, 512, dtype=torch.bfloat16), t(2, 128)
    table, off, vis = t(1, 4, dtype=torch.int32), t(2, dtype=torch.int32), t(2, dtype=torch.int32)
    pool, ws = t(4, 64, 576, dtype=torch.uint8), t(256, dtype=torch.uint8)
    good = dict(q=q, kv_pool=pool, page_table=table, q_offsets=off, q_vis=vis, B=1, sinks=0, window=5, scale=1.0, out=out,
                lse=lse, ws=ws, kv_scales=t(4, 4))
    bad = [dict(q=q.float()), dict(q=t(2, 128, 512, dtype=torch.bfloat16)), dict(out=out.float()), dict(lse=t(2, 64)),
           dict(kv_pool=pool.to(torch.bfloat16)), dict(kv_scales=None), dict(kv_scales=t(4, 5)), dict(kv_scales=t(3, 4)),
           dict(page_table=t(2, 4, dtype=torch.int32)), dict(q_offsets=t(3, dtype=torch.int32)),
           dict(q_vis=t(2, dtype=torch.int64)), {}]
    for over in bad:                                   # the last: host tensors
        with pytest.raises(ValueError):
            dsa.dsa_mla_decode_sinks(**{**good, **over})
    del good["sinks"], good["window"]
    for over in [dict(idx=t(2, 9)), dict(idx=t(3, 9, dtype=torch.int32)), dict(idx=t(2, 9, dtype=torch.int32))]:
        with pytest.raises(ValueError):
            dsa.dsa_sparse_mla_decode_fp8_block(**{**good, **over})


def test_reference_rounding_matches_the_type():
    """The tests' own e4m3 rounding against torch's, over every bf16 value in range."""
    v = torch.arange(0, 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    v = v[(v <= 448.0)]
    assert torch.equal(e4m3_round(v), v.float().to(torch.float8_e4m3fn).double())
    assert torch.equal(e4m3_round(-v), (-v).float().to(torch.float8_e4m3fn).double())
    assert float(e4m3_round(torch.tensor([1e30], dtype=torch.float64))) == 448.0
    assert torch.isnan(e4m3_round(torch.tensor([math.nan, math.inf], dtype=torch.float64))).all()
