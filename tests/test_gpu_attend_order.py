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


def step(heads=128, users=40):
    """One decode step's arrays: an append of one token a user, and the attention over the window behind it."""
    lens = [200 + 5 * b for b in range(users)]
    cache = Cache(lens, 64, True, 64, seed=9)
    g = cache.g
    s = dict(cache=cache, x=torch.randn(users, D, device=DEV, generator=g).to(torch.bfloat16),
             q=torch.randn(users, heads, D, device=DEV, generator=g).to(torch.bfloat16),
             off=cache.offsets([1] * users), vis=torch.tensor(lens, dtype=torch.int32, device=DEV),
             freq=torch.rand(32, device=DEV, generator=g), ws=dsa.attend_workspace(heads),
             out=torch.empty(users, heads, DV, dtype=torch.bfloat16, device=DEV), lse=torch.empty(users, heads, device=DEV))
    s["mine"] = torch.zeros_like(s["q"])
    s["tokens"] = torch.zeros_like(s["x"])
    return s


def append(s):
    c = s["cache"]
    dsa.dsa_latent_append(s["tokens"][:, :DV], s["tokens"][:, DV:], s["freq"], c.pool, c.table, s["off"], s["vis"],
                          s["off"].numel() - 1, s["ws"], kv_scales=c.scales)


def attend(s):
    c = s["cache"]
    dsa.dsa_mla_decode_sinks(s["mine"], c.pool, c.table, s["off"], s["vis"], s["off"].numel() - 1, 4, 150, SCALE, s["out"],
                             s["lse"], s["ws"], kv_scales=c.scales)


def expected(s):
    """The same step on copies, idle between its parts."""
    t = dict(s, out=s["out"].clone(), lse=s["lse"].clone(), ws=dsa.attend_workspace(s["q"].shape[1]))
    t["mine"], t["tokens"] = s["q"].clone(), s["x"].clone()
    pool, scales = s["cache"].pool.clone(), s["cache"].scales.clone()
    for part in (append, attend):
        torch.cuda.synchronize()
        part(t)
    torch.cuda.synchronize()
    s["cache"].pool.copy_(pool)
    s["cache"].scales.copy_(scales)
    return t["out"], t["lse"]


def busy(ms):
    torch.cuda._sleep(int(ms * 1.9e6))


@pytest.mark.parametrize("captured", [False, True])
def test_attention_behind_work_of_another_stream(captured):
    """Queries are copied on one stream and tokens appended on another; the attention waits for both by an event."""
    s = step()
    want = expected(s)
    other = torch.cuda.Stream()

    def both():
        main = torch.cuda.current_stream()
        other.wait_stream(main)
        with torch.cuda.stream(other):
            busy(1)                                              # the event comes long after the copy below
            s["tokens"].copy_(s["x"])
            append(s)
        s["mine"].copy_(s["q"])
        main.wait_stream(other)
        attend(s)

    pool, scales = s["cache"].pool.clone(), s["cache"].scales.clone()
    if captured:
        both()                                                   # sets the kernels' attributes before the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both()
    for _ in range(3):
        s["cache"].pool.copy_(pool)
        s["cache"].scales.copy_(scales)
        s["mine"].zero_()
        s["tokens"].zero_()
        torch.cuda.synchronize()
        graph.replay() if captured else both()
        torch.cuda.synchronize()
        assert torch.equal(s["out"], want[0]) and torch.equal(s["lse"], want[1])
    dsa.dsa_check_error(s["ws"])


@pytest.mark.parametrize("before", ["memcpy", "memset", "host copy"])
def test_attention_captured_behind_copies(before):
    """The operation ahead of the attention in a captured stream is no kernel."""
    s = step(64)
    s["tokens"].copy_(s["x"])
    want = expected(s)
    append(s)
    host = s["vis"].cpu().pin_memory()
    extra = torch.zeros(1 << 20, device=DEV)
    attend(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        busy(0.2)
        s["mine"].copy_(s["q"])
        if before == "memcpy":
            extra[:1 << 19].copy_(extra[1 << 19:])
        elif before == "memset":
            extra.zero_()
        else:
            s["vis"].copy_(host, non_blocking=True)
        attend(s)
    s["mine"].zero_()
    if before == "host copy":
        s["vis"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    dsa.dsa_check_error(s["ws"])
    assert torch.equal(s["out"], want[0]) and torch.equal(s["lse"], want[1])
